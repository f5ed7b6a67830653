// output = BF16(act(x W^T + bias) + residual), on the 5th-generation tensor cores.
//
// Three forms.  One token: no tensor core, below.  Few tiles: a CTA takes 128 features
// (rows of W) and up to 256 tokens; the product's M is the features and its N the
// tokens, so that few tokens cost few columns.  One warp loads 64-wide tiles of both with
// TMA through a ring, one issues the products into TMEM.  A cluster of CTAs may share a
// tile: each sums a range of the inner dimension, and the sums are joined through
// distributed shared memory, 8 features a thread, in the order of the ranges.  Many
// tiles: below.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <type_traits>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_linear_tiles.h"
#include "kda_rows.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace linear {

using namespace rows;

constexpr int kThreads = 256;                    // TMA in warp 4, products in warp 5
constexpr int kM = 128, kK = 64;                 // features of a tile, inner of a block
constexpr int kMostN = 256;
constexpr int kMostStages = 10;
constexpr int kATile = kM * kK * 2;
// Bytes of the ring: all that an SM has, or half, where CTAs are more than SMs and 4
// stages fit, so that one's loads run while another starts or ends.
constexpr int kHalfRing = 96 * 1024, kRing = 192 * 1024;

struct Params {
  int rows, inner, outer, act;
  int tile_n, tiles_m, stages, ring, blocks, split;      // blocks: of kK along inner
  int64_t r_stride, o_stride;
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *output;
  int32_t *err;
};

struct Ctrl {
  uint64_t full[kMostStages], empty[kMostStages], done;
  uint32_t tmem, abort;
};

constexpr int smem_of(int ring) { return ring + 1024 + static_cast<int>(sizeof(Ctrl)); }
static_assert(smem_of(kRing) <= 232448, "shared memory of one CTA");

// y (1 + erf(y / sqrt 2)) / 2 = max(y, 0) - |y| erfc(x) / 2 with x = |y| / sqrt 2 and
// erfc(x) = exp(-x^2) t P(t), t = 1 / (1 + x / 2): P is the least-squares fit of relative
// errors at 400 Chebyshev points of 0 <= x <= 10, degree 8, 5e-8 (with FP32's roundings
// 1.8e-7); behind x = 9.4 the exponential is 0, and |y| is kept to 20 beside it, so that of
// infinities these are infinity and 0.  About 15 instructions (the library's erfc: 9159 x
// 256 x 4096 98 us instead of 39).
__device__ __forceinline__ float gelu(float y) {
  const float a = fabsf(y);
  const float t = rcp_approx(__fmaf_rn(a, 0.35355339f, 1.0f));
  float h = -3.005435318e-02f;
  h = __fmaf_rn(h, t, 1.447230577e-01f);
  h = __fmaf_rn(h, t, -2.484147847e-01f);
  h = __fmaf_rn(h, t, 1.442575753e-01f);
  h = __fmaf_rn(h, t, -1.669950970e-02f);
  h = __fmaf_rn(h, t, 1.026802137e-01f);
  h = __fmaf_rn(h, t, 1.212396920e-01f);
  h = __fmaf_rn(h, t, 1.412269175e-01f);
  h = __fmaf_rn(h, t, 1.410411745e-01f);
  const float e = exp2_approx(y * y * -0.72134752f);       // exp(-y^2 / 2)
  return __fmaf_rn(-fminf(a, 20.0f), h * t * e, fmaxf(y, 0.0f));
}

__device__ __forceinline__ float activated(float y, int act) {
  if (act == KDA_ACT_SILU) return silu_approx(y);
  if (act == KDA_ACT_GELU) return gelu(y);
  if (act == KDA_ACT_SOFTPLUS) return softplus(y);
  return y;
}

__device__ __forceinline__ void ld_cluster(uint32_t from, float &a, float &b, float &c, float &d) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(a), "=f"(b), "=f"(c), "=f"(d)
               : "r"(from)
               : "memory");
}

// The epilogue of 8 features of a token (fewer at the end of the row).
template <int kAct>
__device__ __forceinline__ void finish(const Params &p, int64_t row, int feature, const float (&bias)[8],
                                       const uint4 &residual, float (&y)[8]) {
  const int left = p.outer - feature;
  float add[8];
  unpack8(residual, add);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = activated(y[e] + bias[e], kAct) + add[e];
  __nv_bfloat16 *out = p.output + row * p.o_stride + feature;
  if (left >= 8) {
    *reinterpret_cast<uint4 *>(out) = pack8(y);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < left) out[e] = __float2bfloat16_rn(y[e]);
  }
}
// 8 BF16 of a row, zeros behind its end.
__device__ __forceinline__ uint4 vector_of(const __nv_bfloat16 *from, int left) {
  if (left >= 8) return *reinterpret_cast<const uint4 *>(from);
  const uint16_t *at = reinterpret_cast<const uint16_t *>(from);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < left) w[e / 2] |= static_cast<uint32_t>(at[e]) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kAct>
__global__ void __launch_bounds__(kThreads, 2)
    product_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ uint8_t raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Ctrl &c = *reinterpret_cast<Ctrl *>(ring + p.ring);
  const int warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int feature0 = tile % p.tiles_m * kM, row0 = tile / p.tiles_m * p.tile_n;
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
  follow();

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
  const int rows = min(p.tile_n, p.rows - row0);
  float *part = reinterpret_cast<float *>(ring);           // [token][feature]
  __syncthreads();
  if (warp < 4) {
    for (int n = 0; n < rows; n += 32) {
      uint32_t r[32];
      tc_ld(tmem + (static_cast<uint32_t>(warp * 32) << 16) + n, r);
      tc_wait_ld(r);
      float *to = part + n * kM + threadIdx.x;
      if (n + 32 <= rows) {
#pragma unroll
        for (int i = 0; i < 32; ++i) to[i * kM] = __uint_as_float(r[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (n + i < rows) to[i * kM] = __uint_as_float(r[i]);
      }
    }
  }
  if (p.split == 1)
    __syncthreads();
  else
    cluster_sync_all();
  if (ok) {
    // 16 threads a token; this CTA's share of them
    const int first = static_cast<int>(static_cast<int64_t>(rows) * rank / p.split);
    const int last = static_cast<int>(static_cast<int64_t>(rows) * (rank + 1) / p.split);
    const int at = threadIdx.x % 16 * 8, feature = feature0 + at, left = p.outer - feature;
    if (left > 0) {
      float bias[8];
      unpack8(p.bias ? vector_of(p.bias + feature, left) : make_uint4(0, 0, 0, 0), bias);
      // kMany tokens in flight
      auto join = [&](int n0, auto many) {
        constexpr int kMany = decltype(many)::value, kStep = kThreads / 16;
        float y[kMany][8];
        uint4 residual[kMany];
#pragma unroll
        for (int u = 0; u < kMany; ++u) {
          const float *mine = part + (n0 + u * kStep) * kM + at;
          if (p.split == 1) {
            const float4 lo = reinterpret_cast<const float4 *>(mine)[0];
            const float4 hi = reinterpret_cast<const float4 *>(mine)[1];
            y[u][0] = lo.x, y[u][1] = lo.y, y[u][2] = lo.z, y[u][3] = lo.w;
            y[u][4] = hi.x, y[u][5] = hi.y, y[u][6] = hi.z, y[u][7] = hi.w;
          } else {
            float v[8][8];                                   // all in flight, then added in order
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < p.split) {
                const uint32_t from = cluster_map(mine, q);
                ld_cluster(from, v[q][0], v[q][1], v[q][2], v[q][3]);
                ld_cluster(from + 16, v[q][4], v[q][5], v[q][6], v[q][7]);
              }
#pragma unroll
            for (int e = 0; e < 8; ++e) y[u][e] = v[0][e];
#pragma unroll
            for (int q = 1; q < 8; ++q)
              if (q < p.split)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[u][e] += v[q][e];
          }
          residual[u] = p.residual
                            ? vector_of(p.residual + static_cast<int64_t>(row0 + n0 + u * kStep) * p.r_stride +
                                            feature, left)
                            : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kMany; ++u)
          finish<kAct>(p, row0 + n0 + u * kStep, feature, bias, residual[u], y[u]);
      };
      int n = first + threadIdx.x / 16;
      if (p.split == 1)
        for (; n + 3 * (kThreads / 16) < last; n += 4 * (kThreads / 16))
          join(n, std::integral_constant<int, 4>());
      for (; n < last; n += kThreads / 16) join(n, std::integral_constant<int, 1>());
    }
  }
  __syncwarp();
  if (p.split > 1) cluster_sync_all();                     // what others read stays until they did
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

// ------------------------------------------------------------------- one token
//
// A matrix times a vector, bound by W's bytes: a warp takes 2 features over a slice of the
// inner dimension, 8 values a lane and load, 8 loads in flight, in FP32; the token waits
// in shared memory.  The 8 warps of a CTA are slices of the same features where features
// are few, joined in shared memory in order.  No barriers, tensor memory or tensor maps
// have to be set up first: 4096 x 1024 3.3 us in a graph (the clusters above 4.8), 4096 x
// 16384 22.1 (21.9), 7168 x 7168 18.1 (18.6).  With 2 tokens the same is no faster than
// they are, with 4 slower (the tokens' values are unpacked for every feature).
constexpr int kOneThreads = 256, kOneWarps = kOneThreads / 32, kOneMost = 32768;   // values

template <int kAct>
__global__ void __launch_bounds__(kOneThreads)
    one_kernel(const __grid_constant__ Params p, const __nv_bfloat16 *x, const __nv_bfloat16 *w,
               int64_t w_stride) {
  constexpr int kFeatures = 2, kAhead = 4;
  extern __shared__ __align__(16) uint8_t raw[];
  uint4 *token = reinterpret_cast<uint4 *>(raw);
  __shared__ float part[kOneWarps][kFeatures];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = kOneWarps / p.split;                   // pairs of features of a CTA
  const int feature0 = (blockIdx.x * per + warp / p.split) * kFeatures, slice = warp % p.split;
  // vectors of 8 of the slice
  const int vectors = (p.inner + 7) / 8, begin = vectors * slice / p.split;
  const int end = feature0 < p.outer ? vectors * (slice + 1) / p.split : 0;
  const __nv_bfloat16 *row[kFeatures];
#pragma unroll
  for (int f = 0; f < kFeatures; ++f) row[f] = w + min(feature0 + f, p.outer - 1) * w_stride;
  uint4 in[kAhead][kFeatures];
  auto load = [&](int v0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int v = v0 + 32 * u, left = v < end ? p.inner - 8 * v : 0;
#pragma unroll
      for (int f = 0; f < kFeatures; ++f)
        in[u][f] = left >= 8 ? __ldcs(reinterpret_cast<const uint4 *>(row[f] + 8 * v))
                             : vector_of(row[f] + 8 * v, left);
    }
  };
  follow();
  load(begin + lane);
  for (int v = threadIdx.x; v < vectors; v += kOneThreads)
    token[v] = vector_of(x + 8 * v, p.inner - 8 * v);
  __syncthreads();
  float sum[kFeatures] = {0.0f, 0.0f};
  for (int v0 = begin + lane; v0 < end; v0 += 32 * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (v0 + 32 * u >= end) break;
      float a[kFeatures][8], b[8];
      unpack8(token[v0 + 32 * u], b);
#pragma unroll
      for (int f = 0; f < kFeatures; ++f) {
        unpack8(in[u][f], a[f]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[f] = __fmaf_rn(a[f][e], b[e], sum[f]);
      }
    }
    if (v0 + 32 * kAhead < end) load(v0 + 32 * kAhead);
  }
#pragma unroll
  for (int f = 0; f < kFeatures; ++f) sum[f] = warp_sum(sum[f]);
  if (lane < kFeatures) part[warp][lane] = lane == 0 ? sum[0] : sum[1];
  __syncthreads();
  const int pair_of = threadIdx.x / kFeatures, i = threadIdx.x % kFeatures;
  const int feature = (blockIdx.x * per + pair_of) * kFeatures + i;
  if (pair_of < per && feature < p.outer) {
    float y = 0.0f;
    for (int q = 0; q < p.split; ++q) y += part[pair_of * p.split + q][i];
    y = activated(y + (p.bias ? __bfloat162float(p.bias[feature]) : 0.0f), kAct);
    if (p.residual) y += __bfloat162float(p.residual[feature]);
    p.output[feature] = __float2bfloat16_rn(y);
  }
}

typedef void (*OneKernel)(const Params, const __nv_bfloat16 *, const __nv_bfloat16 *, int64_t);

static int launch_one(const kda_linear_args *a, Params &p, int dev, int sms, cudaStream_t stream) {
  const int64_t pairs = (static_cast<int64_t>(a->outer) + 1) / 2;
  // slices until every SM has two CTAs, of 256 values at least
  p.split = 1;
  while (p.split < kOneWarps && pairs * p.split < 2ll * sms * kOneWarps && a->inner >= 512 * p.split)
    p.split *= 2;
  static const OneKernel kernels[4] = {one_kernel<KDA_ACT_NONE>, one_kernel<KDA_ACT_SILU>,
                                       one_kernel<KDA_ACT_GELU>, one_kernel<KDA_ACT_SOFTPLUS>};
  static std::atomic<bool> done[4][kMaxDevices];
  const OneKernel kernel = kernels[p.act];
  if (!set_smem_limit_once(done[p.act], dev, reinterpret_cast<const void *>(kernel), 2 * kOneMost))
    return KDA_ERR_LAUNCH;
  const int64_t grid = (pairs * p.split + kOneWarps - 1) / kOneWarps;
  return launch_following(kernel, grid, kOneThreads, (a->inner + 7) / 8 * 16, 0, stream, p,
                          static_cast<const __nv_bfloat16 *>(a->x),
                          static_cast<const __nv_bfloat16 *>(a->weight), a->w_stride)
             ? KDA_SUCCESS
             : KDA_ERR_LAUNCH;
}

// ------------------------------------------------------------------ many tokens
//
// Tiles of 256 tokens x 256 features, a pair of CTAs on two SMs that walks its tiles.
// A CTA holds 128 tokens' sums and loads their rows and 128 features' of W; a product
// takes the tokens of both and the features of both, so that a CTA loads 32 KiB where
// one alone would load 48 for as many products (128 x 256 tiles of single CTAs: 323 us
// where pairs take 283, 9159 x 4096 x 7168; their loads came in at 70 bytes a cycle and
// SM).  One warp loads, one of the first CTA issues the products, 16 warps take
// the sums of the tile before (the two halves of TMEM hold a tile each) through swizzled
// shared memory, 64 features at a time, the residual in by TMA and the output out by
// TMA, which clips it (to whole vectors of 8: a copy that ends inside one wrote an
// element behind; threads store the last few features).
constexpr int kTileStages = 5;
constexpr int kTileThreads = 640;                // TMA, products, 2 idle; 16 epilogue warps
constexpr int kTileStage = (kTileRows + kTileCols) / 2 * kK * 2;     // of a CTA
constexpr int kChunk = kChunkRows * kChunkCols * 2;                  // bytes of a warp's part of a tile

struct TileCtrl {
  uint64_t full[kTileStages], empty[kTileStages], sums_full[2], sums_empty[2], residual[16];
  uint32_t tmem, abort;
};
constexpr int kTileSmem = kTileStages * kTileStage + 16 * kChunk + 1024 + sizeof(TileCtrl);
static_assert(kTileSmem <= 232448, "shared memory of one CTA");

// The pair's forms of a load (whose bytes count on the first CTA's barrier), a product,
// a commit (which arrives in both CTAs) and an arrival on the first CTA's barrier.
__device__ __forceinline__ void pair_load(void *dst, const CUtensorMap *map, int x, int y,
                                          uint32_t bar_in_first) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar_in_first)
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Relaxed: it says that TMEM was read, which tcgen05's fences order.  (A release waited for
// the output's copy, too: 1500 cycles, 9159 x 256 x 4096 25.1 instead of 19.3 us.)
__device__ __forceinline__ void arrive_in(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int kAct>
__global__ void __launch_bounds__(kTileThreads, 1) __cluster_dims__(2, 1, 1)
    tile_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap xmap,
                const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap rmap,
                const __grid_constant__ CUtensorMap omap) {
  extern __shared__ uint8_t raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *chunks = ring + kTileStages * kTileStage;
  TileCtrl &c = *reinterpret_cast<TileCtrl *>(chunks + 16 * kChunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair0 = blockIdx.x >> 1, pairs = gridDim.x >> 1;
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
      mbar_init(&c.sums_empty[i], 32);           // both CTAs' warps
    }
    for (int i = 0; i < 16; ++i) mbar_init(&c.residual[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&c.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                              // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  follow();

  if (warp == 0) {
    if (elect_one()) {
      int s = 0, phase = 1;
      bool ok = true;
      for (int n = pair0; n < tiles && ok; n += pairs) {
        const Tile tile = tile_of(n, tiles_m, tiles_n);
        for (int k = 0; k < p.blocks; ++k) {
          if (!(ok = wait_phase(&c.empty[s], phase, &c.abort))) break;
          uint8_t *a = ring + s * kTileStage;
          const uint32_t bar = cluster_map(&c.full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&c.full[s], 2 * kTileStage);
          pair_load(a, &xmap, k * kK, tile.row + 128 * rank, bar);
          pair_load(a + kTileStage / 2, &wmap, k * kK, tile.col + 128 * rank, bar);
          if (++s == kTileStages) s = 0, phase ^= 1;
        }
      }
      // the products that still read the ring arrive on barriers of both CTAs
      for (int i = 0; i < kTileStages && ok; ++i) {
        ok = wait_phase(&c.empty[s], phase, &c.abort);
        if (++s == kTileStages) s = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((kTileCols >> 3) << 17) |
                                 ((kTileRows >> 4) << 24);
      int s = 0, phase = 0, i = 0;
      bool ok = true;
      for (int n = pair0; n < tiles && ok; n += pairs, ++i) {
        const int half = i & 1;
        if (!wait_phase(&c.sums_empty[half], ((i >> 1) & 1) ^ 1, &c.abort)) break;
        tc_fence_after();
        const uint32_t d = tmem + half * kTileCols;
        for (int k = 0; k < p.blocks; ++k) {
          if (!(ok = wait_phase(&c.full[s], phase, &c.abort))) break;
          tc_fence_after();
          const uint32_t a = smem_addr(ring + s * kTileStage);
          const uint64_t da = desc_k_major(a), db = desc_k_major(a + kTileStage / 2);
#pragma unroll
          for (int j = 0; j < kK / 16; ++j) pair_mma(d, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
          pair_commit(&c.empty[s]);
          if (++s == kTileStages) s = 0, phase ^= 1;
        }
        pair_commit(&c.sums_full[half]);
      }
    }
  } else if (warp >= 4) {
    // Each warp takes 32 tokens x 64 features of a tile through a buffer of its own, and
    // waits for none of the others.  16 warps, as a chunk is a long chain for one warp
    // (TMEM, arithmetic, shared memory, a fence, a copy: 3.1k cycles where a thin tile's
    // products take 2k); 8 warps with two chunks each took 33 us where 16 took 27.
    const int w4 = warp & 3, group = (warp - 4) >> 2;
    const bool leader = lane == 0;
    uint8_t *const chunk = chunks + (warp - 4) * kChunk, *const mine = chunk + lane * 128;
    uint64_t *const residual = &c.residual[warp - 4];
    const Chunks chunks_of = {p.rows, p.outer, pair0, pairs, 128 * rank + kChunkRows * w4, group * kChunkCols};
    uint32_t loads = 0;
    auto fetch = [&](const Tile &at) {             // a chunk's residual
      if (!leader || !p.residual) return;
      bulk_wait_read(0);                           // the last output has left the buffer
      mbar_arrive_expect_tx(residual, kChunk);
      tma_load(chunk, &rmap, at.col, at.row, residual);
    };
    auto work = [&](int q, const Tile &at, bool there) {
      const int half = q & 1;
      const int left = p.outer - at.col;           // features of the chunk, where fewer than 64
      uint4 bias[4];                               // of the next 32 features
      auto ahead = [&](int z) {
        if (p.bias && there)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            bias[g] = vector_of(p.bias + at.col + 32 * z + 8 * g, left - 32 * z - 8 * g);
      };
      ahead(0);
      bool ok = wait_phase(&c.sums_full[half], (q >> 1) & 1, &c.abort);
      tc_fence_after();
      if (p.residual && there) ok &= wait_phase(residual, loads++ & 1, &c.abort);
      if (leader) bulk_wait_read(0);               // the last output has left the buffer
      if (!__all_sync(0xffffffffu, ok)) return false;
      const uint32_t from =
          tmem + (static_cast<uint32_t>(w4 * 32) << 16) + half * kTileCols + group * 64;
#pragma unroll
      for (int z = 0; z < 2; ++z) {                // 32 features
        uint32_t r[32];
        tc_ld(from + 32 * z, r);
        tc_wait_ld(r);
        if (z == 1) {
          tc_fence_before();
          __syncwarp();
          if (leader) arrive_in(cluster_map(&c.sums_empty[half], 0));
        }
        if (!there) continue;
        if (p.bias) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float add[8];
            unpack8(bias[g], add);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              r[8 * g + e] = __float_as_uint(__uint_as_float(r[8 * g + e]) + add[e]);
          }
          if (z == 0) ahead(1);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e)
          r[e] = __float_as_uint(activated(__uint_as_float(r[e]), kAct));
        if (p.residual) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float add[8];
            unpack8(*reinterpret_cast<const uint4 *>(mine + (((4 * z + g) ^ (lane & 7)) << 4)), add);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              r[8 * g + e] = __float_as_uint(__uint_as_float(r[8 * g + e]) + add[e]);
          }
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<uint4 *>(mine + (((4 * z + g) ^ (lane & 7)) << 4)) =
              make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
        const int end = left - 32 * z;             // the output ends inside a vector of these 32
        if (end > 0 && end < 32 && (end & 7) && at.row + lane < p.rows) {
          uint16_t *out = reinterpret_cast<uint16_t *>(p.output) + (at.row + lane) * p.o_stride + at.col + 32 * z;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= (end & ~7) && e < end) out[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        }
      }
      if (!there) return true;
      fence_proxy_async_smem();
      __syncwarp();
      if (leader) {
        tma_store(&omap, at.col, at.row, chunk);
        bulk_commit();
      }
      return true;
    };
    walk_chunks(chunks_of, fetch, work);
    if (leader) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                              // nothing comes from the other CTA any more
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
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

typedef void (*TileKernel)(const Params, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                           const CUtensorMap);

// Clusters of `cluster` such CTAs that run at a time (fewer than the SMs' number over it,
// where SMs have no partners left).
static int clusters_of(std::atomic<int> (&known)[kMaxDevices], int dev, const void *kernel, int cluster,
                       int threads, int smem) {
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();                          // (not the launch's)
      return 0;
    }
    known[dev].store(n, std::memory_order_release);
  }
  return n;
}

static int launch_tiles(const kda_linear_args *a, const Params &p, int dev, int sms, cudaStream_t stream) {
  const int64_t tiles = static_cast<int64_t>((a->rows + kTileRows - 1) / kTileRows) *
                        ((a->outer + kTileCols - 1) / kTileCols);
  if (tiles > 0x7fffffffll - sms) return KDA_ERR_SHAPE;
  CUtensorMap x, w, r = {}, o;
  if (!rows_map(&x, a->x, a->inner, a->rows, a->x_stride, 128, dev) ||
      !rows_map(&w, a->weight, a->inner, a->outer, a->w_stride, 128, dev) ||
      !rows_map(&o, a->output, a->outer / 8 * 8, a->rows, a->o_stride, 32, dev) ||
      (a->residual && !rows_map(&r, a->residual, a->outer, a->rows, a->r_stride, 32, dev)))
    return KDA_ERR_LAUNCH;
  static const TileKernel kernels[4] = {tile_kernel<KDA_ACT_NONE>, tile_kernel<KDA_ACT_SILU>,
                                        tile_kernel<KDA_ACT_GELU>, tile_kernel<KDA_ACT_SOFTPLUS>};
  static std::atomic<bool> done[4][kMaxDevices];
  const TileKernel kernel = kernels[p.act];
  if (!set_smem_limit_once(done[p.act], dev, reinterpret_cast<const void *>(kernel), kTileSmem))
    return KDA_ERR_LAUNCH;
  static std::atomic<int> known[kMaxDevices];
  const int pairs = clusters_of(known, dev, reinterpret_cast<const void *>(kernel), 2, kTileThreads, kTileSmem);
  if (pairs < 1) return KDA_ERR_LAUNCH;
  return launch_following(kernel, 2 * (tiles < pairs ? tiles : pairs), kTileThreads, kTileSmem, 0, stream,
                          p, x, w, r, o)
             ? KDA_SUCCESS
             : KDA_ERR_LAUNCH;
}

typedef void (*ProductKernel)(const Params, const CUtensorMap, const CUtensorMap);

// Which form and layout: the cheapest by a model of the time in us, fitted to 36 shapes
// with up to 13 layouts each (what it takes is within 3% of the best of them; a shape of
// 2000 x 104 x 104 within 21%).  Few tiles: a CTA streams a block of the inner dimension at
// 140 KB a us or in its products' time, W comes at 7.5 MB a us at most (a third more for
// every time it is read again), a CTA starts and ends in 1.55 + 0.02 a token (a third of it
// hidden where two share an SM), and a join costs by its ranks and tokens.  Ranks are powers
// of two: clusters of 3, 5, 6 and 7 leave SMs idle (300 x 8192 x 640 18.1 us with one, 11.8
// with 4), and 8 some (128 x 16384 x 512 with 16 clusters of 8, which do not all run at once,
// 18.0 us, with 12 10.7).  Pairs: 0.3 a block, 1.4 a tile at least.  tile_n 0: pairs.
struct Plan {
  int tile_n, split;
};
static Plan plan_of(int rows, int blocks, int inner, int outer, int sms, int eights, int path) {
  const int64_t tiles_m = (outer + kM - 1) / kM;
  const double weights = 2.0 * inner * outer / 7.5e6;
  Plan best = {0, 1};
  double least = 1e300;
  if (path == 2) return best;
  if (path == 0 && outer >= 8 && rows > 64) {
    const int64_t tiles = static_cast<int64_t>((rows + kTileRows - 1) / kTileRows) *
                          ((outer + kTileCols - 1) / kTileCols);
    const double tile = blocks * 0.3 > 1.4 ? blocks * 0.3 : 1.4;
    least = static_cast<double>((tiles + sms / 2 - 1) / (sms / 2)) * tile + 4.9;
  }
  for (int tile_n = 16; tile_n <= kMostN; tile_n += tile_n < 64 ? 16 : 32) {
    if (tile_n - 32 >= rows) break;
    const int64_t tiles = tiles_m * ((rows + tile_n - 1) / tile_n);
    const double bytes = (kATile + tile_n * kK * 2) / 140e3;
    const double block = bytes > 0.00087 * tile_n ? bytes : 0.00087 * tile_n;
    for (int split = 1; split <= (eights > 0 ? 8 : 4) && split <= blocks; split *= 2) {
      const int64_t ctas = tiles * split, room = split == 8 ? 8 * eights : sms;
      const int64_t waves = (ctas + room - 1) / room;
      const double ends = (1.55 + 0.02 * tile_n) * (ctas > sms && tile_n <= 64 ? 0.68 : 1.0);
      double stream = static_cast<double>(waves) * ((blocks + split - 1) / split) * block;
      const double read = weights * (1.0 + 0.32 * ((rows - 1) / tile_n));
      if (stream < read) stream = read;
      const double join = split > 1 ? 0.9 + (split - 1) * 0.005 * tile_n : 0.0;
      const double cost = stream + static_cast<double>(waves) * (ends + join) + 0.3;
      if (cost < least) {
        least = cost;
        best = {tile_n, split};
      }
    }
  }
  return best;
}

static int run(const kda_linear_args *a, int path, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  if (a->rows < 0 || a->inner < 1 || a->outer < 0 || a->rows > kMostRows || a->inner > kMostRows ||
      a->outer > kMostRows)
    return KDA_ERR_SHAPE;
  if (!stride_ok(a->x_stride, a->inner) || !stride_ok(a->w_stride, a->inner) ||
      !stride_ok(a->o_stride, a->outer) || (a->residual && !stride_ok(a->r_stride, a->outer)))
    return KDA_ERR_SHAPE;
  if (a->activation < KDA_ACT_NONE || a->activation > KDA_ACT_SOFTPLUS) return KDA_ERR_ACTIVATION;
  if (path < 0 || path > 2) return KDA_ERR_PATH;
  if (a->rows == 0 || a->outer == 0) return KDA_SUCCESS;
  if (path == 2 && a->outer < 8) return KDA_ERR_SHAPE;   // (an output's tensor map of whole vectors)
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
  if (path == 0 && a->rows == 1 && a->inner <= kOneMost) return launch_one(a, p, dev, df.sms, stream);
  p.blocks = (a->inner + kK - 1) / kK;
  static const ProductKernel kernels[4] = {product_kernel<KDA_ACT_NONE>, product_kernel<KDA_ACT_SILU>,
                                           product_kernel<KDA_ACT_GELU>, product_kernel<KDA_ACT_SOFTPLUS>};
  static std::atomic<bool> done[4][kMaxDevices];
  const ProductKernel kernel = kernels[p.act];
  if (!set_smem_limit_once(done[p.act], dev, reinterpret_cast<const void *>(kernel), smem_of(kRing)))
    return KDA_ERR_LAUNCH;
  static std::atomic<int> known[kMaxDevices];
  const int eights = clusters_of(known, dev, reinterpret_cast<const void *>(kernel), 8, kThreads, smem_of(kRing));
  const Plan plan = plan_of(a->rows, p.blocks, a->inner, a->outer, df.sms, eights, path);
  if (plan.tile_n == 0) return launch_tiles(a, p, dev, df.sms, stream);
  p.tile_n = plan.tile_n;
  p.split = plan.split;
  const int stage = kATile + p.tile_n * kK * 2;
  p.tiles_m = (a->outer + kM - 1) / kM;
  const int64_t ctas = static_cast<int64_t>(p.tiles_m) * ((a->rows + p.tile_n - 1) / p.tile_n) * p.split;
  if (ctas > 0x7fffffffll) return KDA_ERR_SHAPE;
  const bool few = ctas <= df.sms;
  p.ring = !few && kHalfRing / stage >= 4 ? kHalfRing : kRing;
  p.stages = p.ring / stage;
  if (p.stages > kMostStages) p.stages = kMostStages;
  CUtensorMap w, x;
  if (!rows_map(&w, a->weight, a->inner, a->outer, a->w_stride, kM, dev) ||
      !rows_map(&x, a->x, a->inner, a->rows, a->x_stride, p.tile_n, dev))
    return KDA_ERR_LAUNCH;
  return launch_following(kernel, ctas, kThreads, smem_of(p.ring), p.split, stream, p, w, x) ? KDA_SUCCESS
                                                                                             : KDA_ERR_LAUNCH;
}

}  // namespace linear
}  // namespace kda

extern "C" int kda_linear(const kda_linear_args *args, void *stream) {
  return kda::linear::run(args, 0, static_cast<cudaStream_t>(stream));
}

extern "C" int kda_linear_path(const kda_linear_args *args, int32_t path, void *stream) {
  return kda::linear::run(args, path, static_cast<cudaStream_t>(stream));
}
