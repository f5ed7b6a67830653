// output = BF16(act(x W^T + bias) + residual), on the 5th-generation tensor cores.
//
// A CTA takes 128 features (rows of W) and up to 256 tokens: the product's M is
// the features and its N the tokens, so that few tokens cost few columns, and W is
// read once where 256 tokens suffice.  One warp loads 64-wide tiles of both with
// TMA through a ring, one issues the products into TMEM, four take the sums out.
// Where tiles are fewer than SMs, a cluster of CTAs shares a tile: each sums a
// range of the inner dimension, and the sums are joined through distributed shared
// memory in the order of the ranks.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_rows.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace linear {

using namespace rows;

constexpr int kThreads = 192;                    // 4 epilogue warps, TMA, products
constexpr int kM = 128, kK = 64;                 // features of a tile, inner of a block
constexpr int kMostN = 256;
constexpr int kMostStages = 8;
constexpr int kRing = 200 * 1024;                // bytes of the ring, at most
constexpr int kATile = kM * kK * 2;

struct Params {
  int rows, inner, outer, act;
  int tile_n, stages, blocks, split;             // blocks: of kK along inner
  int64_t r_stride, o_stride;
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *output;
  int32_t *err;
};

struct Ctrl {
  uint64_t full[kMostStages], empty[kMostStages], done;
  uint32_t tmem, abort;
};

constexpr int kSmem = kRing + 1024 + sizeof(Ctrl);
static_assert(kSmem <= 232448, "shared memory of one CTA");

__device__ __forceinline__ float activated(float y, int act) {
  if (act == KDA_ACT_SILU) return silu_approx(y);
  if (act == KDA_ACT_GELU) return 0.5f * y * erfcf(y * -0.7071067812f);
  if (act == KDA_ACT_SOFTPLUS) return softplus(y);
  return y;
}

__device__ __forceinline__ void finish(const Params &p, int row, int feature, float bias, float y) {
  y = activated(y + bias, p.act);
  if (p.residual) y += __bfloat162float(p.residual[row * p.r_stride + feature]);
  p.output[row * p.o_stride + feature] = __float2bfloat16_rn(y);
}

__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ uint8_t raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Ctrl &c = *reinterpret_cast<Ctrl *>(ring + kRing);
  const int warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.split, feature0 = blockIdx.x / p.split * kM;
  const int row0 = blockIdx.y * p.tile_n;
  const int stage_bytes = kATile + p.tile_n * kK * 2;
  const int begin = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / p.split);
  const int end = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / p.split);
  if (threadIdx.x == 0) {
    c.abort = 0;
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.empty[i], 1);
    }
    mbar_init(&c.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  uint32_t columns = 32;
  while (columns < static_cast<uint32_t>(p.tile_n)) columns *= 2;
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&c.tmem)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  if (warp == 4) {
    if (elect_one()) {
      for (int k = begin, s = 0, phase = 0; k < end; ++k) {
        if (k - begin >= p.stages && !wait_phase(&c.empty[s], phase ^ 1, &c.abort)) break;
        uint8_t *a = ring + s * stage_bytes;
        mbar_arrive_expect_tx(&c.full[s], stage_bytes);
        tma_load(a, &wmap, k * kK, feature0, &c.full[s]);
        tma_load(a + kATile, &xmap, k * kK, row0, &c.full[s]);
        if (++s == p.stages) s = 0, phase ^= 1;
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    if (elect_one()) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) |
                             (static_cast<uint32_t>(p.tile_n >> 3) << 17) | ((kM >> 4) << 24);
      int s = 0, phase = 0, k = begin;
      for (; k < end; ++k) {
        if (!wait_phase(&c.full[s], phase, &c.abort)) break;
        tc_fence_after();
        const uint32_t a = smem_addr(ring + s * stage_bytes);
        const uint64_t da = desc_k_major(a), db = desc_k_major(a + kATile);
#pragma unroll
        for (int i = 0; i < kK / 16; ++i) tc_mma_ss(tmem, da + 2 * i, db + 2 * i, idesc, k > begin || i > 0);
        tc_commit(&c.empty[s]);
        if (++s == p.stages) s = 0, phase ^= 1;
      }
      tc_commit(&c.done);
    }
    __syncwarp();
  }
  // every warp: what the ring holds is used up behind this
  const bool ok = wait_phase(&c.done, 0, &c.abort);
  tc_fence_after();
  const int feature = feature0 + threadIdx.x;
  const int rows = min(p.tile_n, p.rows - row0);
  if (p.split == 1) {
    if (warp < 4) {
      const float bias =
          p.bias && feature < p.outer ? __bfloat162float(p.bias[feature]) : 0.0f;
      for (int n = 0; n < rows; n += 32) {
        uint32_t r[32];
        tc_ld(tmem + (static_cast<uint32_t>(warp * 32) << 16) + n, r);
        tc_wait_ld(r);
        if (feature < p.outer && ok) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (n + i < rows) finish(p, row0 + n + i, feature, bias, __uint_as_float(r[i]));
        }
      }
    }
  } else {
    float *part = reinterpret_cast<float *>(ring);           // [token][feature]
    __syncthreads();
    if (warp < 4) {
      for (int n = 0; n < rows; n += 32) {
        uint32_t r[32];
        tc_ld(tmem + (static_cast<uint32_t>(warp * 32) << 16) + n, r);
        tc_wait_ld(r);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (n + i < rows) part[(n + i) * kM + threadIdx.x] = __uint_as_float(r[i]);
      }
    }
    cluster_sync_all();
    if (warp < 4 && feature < p.outer && ok) {
      const float bias = p.bias ? __bfloat162float(p.bias[feature]) : 0.0f;
      for (int n = rank; n < rows; n += p.split) {
        float y = 0.0f;
        for (int q = 0; q < p.split; ++q) {
          float v;
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(v)
                       : "r"(cluster_map(part + n * kM + threadIdx.x, q))
                       : "memory");
          y += v;
        }
        finish(p, row0 + n, feature, bias, y);
      }
    }
    cluster_sync_all();
  }
  tc_fence_before();
  __syncthreads();
  if (*static_cast<volatile uint32_t *>(&c.abort)) {
    // copies and products in flight end within microseconds: give them time
    // before the shared memory and TMEM go
    const uint64_t t0 = global_ns();
    for (int i = 0; i < 4096 && global_ns() - t0 < 200000ull; ++i) __nanosleep(1000);
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
    __syncthreads();
  }
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns)
                 : "memory");
  }
}

// ------------------------------------------------------------------ many tokens
//
// Tiles of 128 tokens x 256 features, one CTA an SM that walks its tiles: one warp
// loads, one issues products, two warpgroups take the sums of the tile before (the two
// halves of TMEM hold a tile each) through swizzled shared memory, 64 features at a
// time, the residual in by TMA and the output out by TMA, which clips it (to whole
// vectors of 8: a copy that ends inside one wrote an element behind; threads store the
// last few features).
constexpr int kTileRows = 128, kTileCols = 256, kTileStages = 4;
constexpr int kTileThreads = 384;                // TMA, products, 2 idle; 8 epilogue warps
constexpr int kTileStage = (kTileRows + kTileCols) * kK * 2;
constexpr int kChunk = kTileRows * 64 * 2;       // bytes of 64 features
constexpr int kGroupRows = 16;                   // tiles along the tokens that run side by side

struct TileCtrl {
  uint64_t full[kTileStages], empty[kTileStages], sums_full[2], sums_empty[2], residual[2];
  uint32_t tmem, abort;
};
constexpr int kTileSmem = kTileStages * kTileStage + 2 * kChunk + 1024 + sizeof(TileCtrl);
static_assert(kTileSmem <= 232448, "shared memory of one CTA");

struct Tile {
  int row, col;
};
// Tiles in groups of kGroupRows along the tokens, so that those that run at a time
// share their operands in L2.
__device__ __forceinline__ Tile tile_of(int n, int tiles_m, int tiles_n) {
  const int group = n / (kGroupRows * tiles_n), first = group * kGroupRows;
  const int high = min(kGroupRows, tiles_m - first), at = n - first * tiles_n;
  return Tile{(first + at % high) * kTileRows, at / high * kTileCols};
}

// Named barrier of an epilogue warpgroup that also ORs a predicate.
__device__ __forceinline__ bool group_sync_or(int group, bool pred) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(group + 1)
      : "memory");
  return r != 0;
}

template <int kAct>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap xmap,
                const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap rmap,
                const __grid_constant__ CUtensorMap omap) {
  extern __shared__ uint8_t raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *chunks = ring + kTileStages * kTileStage;
  TileCtrl &c = *reinterpret_cast<TileCtrl *>(chunks + 2 * kChunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_m = (p.rows + kTileRows - 1) / kTileRows;
  const int tiles_n = (p.outer + kTileCols - 1) / kTileCols, tiles = tiles_m * tiles_n;
  if (threadIdx.x == 0) {
    c.abort = 0;
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.sums_full[i], 1);
      mbar_init(&c.sums_empty[i], 8);
      mbar_init(&c.residual[i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&c.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  if (warp == 0) {
    if (elect_one()) {
      int s = 0, phase = 1;
      bool ok = true;
      for (int n = blockIdx.x; n < tiles && ok; n += gridDim.x) {
        const Tile tile = tile_of(n, tiles_m, tiles_n);
        for (int k = 0; k < p.blocks; ++k) {
          if (!(ok = wait_phase(&c.empty[s], phase, &c.abort))) break;
          uint8_t *a = ring + s * kTileStage;
          mbar_arrive_expect_tx(&c.full[s], kTileStage);
          tma_load(a, &xmap, k * kK, tile.row, &c.full[s]);
          tma_load(a + kTileRows * kK * 2, &wmap, k * kK, tile.col, &c.full[s]);
          if (++s == kTileStages) s = 0, phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((kTileCols >> 3) << 17) |
                                 ((kTileRows >> 4) << 24);
      int s = 0, phase = 0, i = 0;
      bool ok = true;
      for (int n = blockIdx.x; n < tiles && ok; n += gridDim.x, ++i) {
        const int half = i & 1;
        if (!wait_phase(&c.sums_empty[half], ((i >> 1) & 1) ^ 1, &c.abort)) break;
        tc_fence_after();
        const uint32_t d = tmem + half * kTileCols;
        for (int k = 0; k < p.blocks; ++k) {
          if (!(ok = wait_phase(&c.full[s], phase, &c.abort))) break;
          tc_fence_after();
          const uint32_t a = smem_addr(ring + s * kTileStage);
          const uint64_t da = desc_k_major(a), db = desc_k_major(a + kTileRows * kK * 2);
#pragma unroll
          for (int j = 0; j < kK / 16; ++j) tc_mma_ss(d, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
          tc_commit(&c.empty[s]);
          if (++s == kTileStages) s = 0, phase ^= 1;
        }
        tc_commit(&c.sums_full[half]);
      }
    }
  } else if (warp >= 4) {
    const int group = (warp - 4) >> 2, w4 = warp & 3, row = w4 * 32 + lane;
    const bool leader = (threadIdx.x & 127) == 0;
    uint8_t *chunk = chunks + group * kChunk, *mine = chunk + row * 128;
    int i = 0, loads = 0;
    for (int n = blockIdx.x; n < tiles; n += gridDim.x, ++i) {
      const Tile tile = tile_of(n, tiles_m, tiles_n);
      const int half = i & 1;
      bool stop = false;
      for (int part = 0; part < 2; ++part) {
        const int col = tile.col + group * 128 + part * 64;
        bool ok = true;
        if (leader) {
          bulk_wait_read(0);                       // the chunk's last output has left
          if (p.residual && col < p.outer) {
            mbar_arrive_expect_tx(&c.residual[group], kChunk);
            tma_load(chunk, &rmap, col, tile.row, &c.residual[group]);
          }
        }
        if (part == 0) {
          ok = wait_phase(&c.sums_full[half], (i >> 1) & 1, &c.abort);
          tc_fence_after();
        }
        uint32_t r[2][32];
        if (group_sync_or(group, !ok)) {           // all of the warpgroup, or none
          stop = true;
          break;
        }
        const uint32_t from =
            tmem + (static_cast<uint32_t>(w4 * 32) << 16) + half * kTileCols + group * 128 + part * 64;
        tc_ld(from, r[0]);
        tc_ld(from + 32, r[1]);
        tc_wait_ld(r[0]);
        tc_wait_ld(r[1]);
        if (part == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.sums_empty[half]);
        }
        if (col >= p.outer) continue;
        if (p.residual) ok = wait_phase(&c.residual[group], loads++ & 1, &c.abort);
#pragma unroll
        for (int g = 0; g < 8; ++g) {              // 8 features, 16 bytes
          float y[8], add[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(r[g >> 2][(g & 3) * 8 + e]);
          if (p.bias && col + 8 * g < p.outer) {
            if (col + 8 * g + 8 <= p.outer) {
              unpack8(__ldg(reinterpret_cast<const uint4 *>(p.bias + col + 8 * g)), add);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                add[e] = col + 8 * g + e < p.outer ? __bfloat162float(p.bias[col + 8 * g + e]) : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += add[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = activated(y[e], kAct);
          uint4 *at = reinterpret_cast<uint4 *>(mine + ((g ^ (row & 7)) << 4));
          if (p.residual) {
            unpack8(*at, add);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] += add[e];
          }
          *at = pack8(y);
          const int left = p.outer - col - 8 * g;
          if (left > 0 && left < 8 && tile.row + row < p.rows) {
            __nv_bfloat16 *out = p.output + (tile.row + row) * p.o_stride + col + 8 * g;
#pragma unroll
            for (int e = 0; e < 7; ++e)
              if (e < left) out[e] = __float2bfloat16_rn(y[e]);
          }
        }
        fence_proxy_async_smem();
        if (group_sync_or(group, !ok)) {
          stop = true;
          break;
        }
        if (leader) {
          tma_store(&omap, col, tile.row, chunk);
          bulk_commit();
        }
      }
      if (stop) break;
    }
    if (leader) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*static_cast<volatile uint32_t *>(&c.abort)) {
    // copies and products in flight end within microseconds: give them time
    // before the shared memory and TMEM go
    const uint64_t t0 = global_ns();
    for (int i = 0; i < 4096 && global_ns() - t0 < 200000ull; ++i) __nanosleep(1000);
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

typedef void (*TileKernel)(const Params, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                           const CUtensorMap);

static int launch_tiles(const kda_linear_args *a, const Params &p, int dev, int sms, cudaStream_t stream) {
  const int64_t tiles = static_cast<int64_t>((a->rows + kTileRows - 1) / kTileRows) *
                        ((a->outer + kTileCols - 1) / kTileCols);
  if (tiles > 0x7fffffffll - sms) return KDA_ERR_SHAPE;
  CUtensorMap x, w, r = {}, o;
  if (!rows_map(&x, a->x, a->inner, a->rows, a->x_stride, kTileRows, dev) ||
      !rows_map(&w, a->weight, a->inner, a->outer, a->w_stride, kTileCols, dev) ||
      !rows_map(&o, a->output, a->outer / 8 * 8, a->rows, a->o_stride, kTileRows, dev) ||
      (a->residual && !rows_map(&r, a->residual, a->outer, a->rows, a->r_stride, kTileRows, dev)))
    return KDA_ERR_LAUNCH;
  static const TileKernel kernels[4] = {tile_kernel<KDA_ACT_NONE>, tile_kernel<KDA_ACT_SILU>,
                                        tile_kernel<KDA_ACT_GELU>, tile_kernel<KDA_ACT_SOFTPLUS>};
  static std::atomic<bool> done[4][kMaxDevices];
  const TileKernel kernel = kernels[p.act];
  if (!set_smem_limit_once(done[p.act], dev, reinterpret_cast<const void *>(kernel), kTileSmem))
    return KDA_ERR_LAUNCH;
  kernel<<<static_cast<int>(tiles < sms ? tiles : sms), kTileThreads, kTileSmem, stream>>>(p, x, w, r, o);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

static int run(const kda_linear_args *a, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  if (a->rows < 0 || a->inner < 1 || a->outer < 0) return KDA_ERR_SHAPE;
  if (!stride_ok(a->x_stride, a->inner) || !stride_ok(a->w_stride, a->inner) ||
      !stride_ok(a->o_stride, a->outer) || (a->residual && !stride_ok(a->r_stride, a->outer)))
    return KDA_ERR_SHAPE;
  if (a->activation < KDA_ACT_NONE || a->activation > KDA_ACT_SOFTPLUS) return KDA_ERR_ACTIVATION;
  if (a->rows == 0 || a->outer == 0) return KDA_SUCCESS;
  if (!a->x || !a->weight || !a->output) return KDA_ERR_NULL_POINTER;
  if (!aligned(a->x, 16) || !aligned(a->weight, 16) || !aligned(a->bias, 16) ||
      !aligned(a->residual, 16) || !aligned(a->output, 16) || !aligned(a->err, 4))
    return KDA_ERR_ALIGNMENT;
  int dev = 0;
  DeviceFacts df;
  if (!current_device(&dev, &df)) return KDA_ERR_DEVICE;
  Params p = {};
  p.rows = a->rows;
  p.inner = a->inner;
  p.outer = a->outer;
  p.act = a->activation;
  p.r_stride = a->r_stride;
  p.o_stride = a->o_stride;
  p.bias = static_cast<const __nv_bfloat16 *>(a->bias);
  p.residual = static_cast<const __nv_bfloat16 *>(a->residual);
  p.output = static_cast<__nv_bfloat16 *>(a->output);
  p.err = a->err;
  p.tile_n = a->rows >= kMostN ? kMostN : (a->rows + 15) / 16 * 16;
  p.blocks = (a->inner + kK - 1) / kK;
  if (a->rows > kMostN && a->outer >= 8) return launch_tiles(a, p, dev, df.sms, stream);
  p.stages = kRing / (kATile + p.tile_n * kK * 2);
  if (p.stages > kMostStages) p.stages = kMostStages;
  const int tiles_m = (a->outer + kM - 1) / kM, tiles_n = (a->rows + p.tile_n - 1) / p.tile_n;
  if (tiles_n > 65535) return KDA_ERR_SHAPE;
  p.split = 1;
  while (p.split < 8 && 2 * p.split * static_cast<int64_t>(tiles_m) * tiles_n <= df.sms &&
         2 * p.split <= p.blocks)
    p.split *= 2;
  CUtensorMap w, x;
  if (!rows_map(&w, a->weight, a->inner, a->outer, a->w_stride, kM, dev) ||
      !rows_map(&x, a->x, a->inner, a->rows, a->x_stride, p.tile_n, dev))
    return KDA_ERR_LAUNCH;
  static std::atomic<bool> done[kMaxDevices];
  if (!set_smem_limit_once(done, dev, reinterpret_cast<const void *>(product_kernel), kSmem))
    return KDA_ERR_LAUNCH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles_m * p.split, tiles_n);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, product_kernel, p, w, x) != cudaSuccess) return KDA_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

}  // namespace linear
}  // namespace kda

extern "C" int kda_linear(const kda_linear_args *args, void *stream) {
  return kda::linear::run(args, static_cast<cudaStream_t>(stream));
}
