// Snapshots: FP32 state pages kept in 8 or 4 bits, and read back.
//
// A group of keys of one value row (8 bits: the row's 128; 4 bits: 32) shares
// one FP32 scale = m / L (m the group's largest magnitude, L = 127 or 7), and
// a code is x / scale to the nearest whole number, ties to even, decided as in
// exact arithmetic: x * (1 / scale), rounded by adding 1.5 * 2^23, gives a candidate
// at most one off, and its residual fma(-code, scale, x) is exact in FP32 (it is a
// multiple of the smaller of the last places of x and scale, and no larger than
// about half a scale; for a code of 0 it is x), so comparing it with scale / 2
// settles the code.  The definition can then be matched code by code.
//
// HBM-bound both ways (a page of 64 KiB against 16.5 or 10 KiB of snapshot).  A
// warp takes 8 rows, lane l the keys 4l .. 4l+3: every row is one 512-byte access
// of the warp, its codes one of 128 (64) bytes, and the rows' loads are in flight
// at once.  GB300, 64 x 32 pages, 8 bits: save 25.6 us = 6.6 TB/s (16 rows a warp:
// 31.5; a division per lane and row besides: 36.5), load 24.7 us; 119 x 64 pages
// read from 4 bits 87 us = 6.6 TB/s.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_host.h"

namespace kda {
namespace snap {

constexpr int kDim = 128;
constexpr int kPage = kDim * kDim;
constexpr int kRows = 8;                         // rows of a warp
constexpr int kWarps = 2;                        // of a CTA
constexpr int kParts = kDim / (kRows * kWarps);  // CTAs of a page

struct Params {
  int heads, num_slots, num_snaps;
  const int32_t *slots, *snaps;
  float4 *state;
  void *codes;
  float *scales;
  int32_t *err;
};

// Entry e's slot and snapshot; false: padding or flagged.
__device__ __forceinline__ bool resolve(const Params &p, int e, int *slot, int *snap) {
  *slot = __ldg(p.slots + e);
  *snap = __ldg(p.snaps + e);
  if (*slot <= 0 || *snap <= 0) return false;
  if (*slot >= p.num_slots || *snap >= p.num_snaps) {
    if (p.err && threadIdx.x == 0) atomicOr(p.err, KDA_DEVERR_SLOT);
    return false;
  }
  return true;
}

// The code of x in the low bits: x / scale to the nearest whole number.  Adding
// 1.5 * 2^23 rounds x * inv to one; `half` is scale / 2.
__device__ __forceinline__ uint32_t quantise(float x, float scale, float half, float inv) {
  constexpr float kMagic = 12582912.0f;
  const float t = __fmaf_rn(x, inv, kMagic);
  uint32_t code = __float_as_uint(t);
  const float r = __fmaf_rn(__fsub_rn(kMagic, t), scale, x);
  if (fabsf(r) >= half) {
    // not the nearest, or a tie: then the even one
    if (fabsf(r) > half || (code & 1u)) code += r > 0.0f ? 1u : 0xFFFFFFFFu;
  }
  return code;
}

template <int kBits>
__global__ void __launch_bounds__(kWarps * 32) save_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = kBits == 8 ? 32 : 8;   // lanes that share a scale
  constexpr int kGroups = 32 / kLanes;          // scales of a row
  constexpr int kOwn = (kRows + kLanes - 1) / kLanes;         // scales a lane works out
  constexpr float kTop = kBits == 8 ? 127.0f : 7.0f;
  const int part = blockIdx.x % kParts, item = blockIdx.x / kParts;
  const int e = item / p.heads, h = item % p.heads;
  const int lane = threadIdx.x & 31, row0 = (part * kWarps + (threadIdx.x >> 5)) * kRows;
  int slot, snap;
  if (!resolve(p, e, &slot, &snap)) return;
  const float4 *page = p.state + (static_cast<int64_t>(slot) * p.heads + h) * (kPage / 4) +
                       row0 * (kDim / 4) + lane;
  const int64_t kept = static_cast<int64_t>(snap) * p.heads + h;
  float4 x[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) x[i] = __ldcs(page + i * (kDim / 4));
  // Every group's largest magnitude, as an integer (an infinity or NaN tops every
  // finite one), and its scale in one lane of the group: the divisions, two of 20
  // instructions, are done once per scale instead of once per lane and row.
  float scale[kOwn], inv[kOwn];
#pragma unroll
  for (int k = 0; k < kOwn; ++k) scale[k] = 0.0f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t m = max(max(__float_as_uint(x[i].x) & 0x7fffffffu, __float_as_uint(x[i].y) & 0x7fffffffu),
                     max(__float_as_uint(x[i].z) & 0x7fffffffu, __float_as_uint(x[i].w) & 0x7fffffffu));
    if (kLanes == 32) {
      m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if ((lane & (kLanes - 1)) == (i & (kLanes - 1))) scale[i / kLanes] = __uint_as_float(m);
  }
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const float top = scale[k];
    const bool bad = !(top <= 3.402823466e38f), small = top < 0x1p-118f;
    scale[k] = bad ? __uint_as_float(0x7fffffffu) : small ? 0.0f : __fdiv_rn(top, kTop);
    inv[k] = bad || small ? 0.0f : __fdiv_rn(1.0f, scale[k]);
    const int i = k * kLanes + (lane & (kLanes - 1));
    if (i < kRows) p.scales[(kept * kDim + row0 + i) * kGroups + lane / kLanes] = scale[k];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int from = (lane & ~(kLanes - 1)) | (i & (kLanes - 1));
    const float s = __shfl_sync(0xffffffffu, scale[i / kLanes], from);
    const float v = __shfl_sync(0xffffffffu, inv[i / kLanes], from);
    const float half = 0.5f * s;
    uint32_t c[4] = {0, 0, 0, 0};
    if (v > 0.0f) {
      c[0] = quantise(x[i].x, s, half, v);
      c[1] = quantise(x[i].y, s, half, v);
      c[2] = quantise(x[i].z, s, half, v);
      c[3] = quantise(x[i].w, s, half, v);
    }
    if (kBits == 8) {
      const uint32_t w =
          __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
      static_cast<uint32_t *>(p.codes)[(kept * kDim + row0 + i) * 32 + lane] = w;
    } else {
      const uint32_t w = (c[0] & 15) | (c[1] & 15) << 4 | (c[2] & 15) << 8 | (c[3] & 15) << 12;
      static_cast<uint16_t *>(p.codes)[(kept * kDim + row0 + i) * 32 + lane] =
          static_cast<uint16_t>(w);
    }
  }
}

template <int kBits>
__global__ void __launch_bounds__(kWarps * 32) load_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = kBits == 8 ? 32 : 8;
  constexpr int kGroups = 32 / kLanes;
  const int part = blockIdx.x % kParts, item = blockIdx.x / kParts;
  const int e = item / p.heads, h = item % p.heads;
  const int lane = threadIdx.x & 31, row0 = (part * kWarps + (threadIdx.x >> 5)) * kRows;
  int slot, snap;
  if (!resolve(p, e, &slot, &snap)) return;
  float4 *page = p.state + (static_cast<int64_t>(slot) * p.heads + h) * (kPage / 4) +
                 row0 * (kDim / 4) + lane;
  const int64_t kept = static_cast<int64_t>(snap) * p.heads + h;
  const float *scales = p.scales + (kept * kDim + row0) * kGroups;
  uint32_t w[kRows];
  float scale[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (kBits == 8)
      w[i] = __ldg(static_cast<const uint32_t *>(p.codes) + (kept * kDim + row0 + i) * 32 + lane);
    else
      w[i] = __ldg(static_cast<const uint16_t *>(p.codes) + (kept * kDim + row0 + i) * 32 + lane);
    scale[i] = __ldg(scales + i * kGroups + lane / kLanes);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = static_cast<float>(static_cast<int32_t>(w[i] << (32 - kBits * (j + 1))) >> (32 - kBits));
    __stcs(page + i * (kDim / 4), make_float4(c[0] * scale[i], c[1] * scale[i], c[2] * scale[i],
                                              c[3] * scale[i]));
  }
}

static bool aligned(const void *q, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(q) & (to - 1)) == 0;
}

static int run(const kda_snapshot_args *a, bool save, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  if (a->count < 0 || a->heads < 0 || a->num_slots < 1 || a->num_snaps < 1 ||
      (a->bits != 8 && a->bits != 4) ||
      static_cast<int64_t>(a->count) * a->heads > 0x7fffffffll / kParts)
    return KDA_ERR_SHAPE;
  if (a->count == 0 || a->heads == 0) return KDA_SUCCESS;
  if (!a->slots || !a->snaps || !a->state || !a->codes || !a->scales) return KDA_ERR_NULL_POINTER;
  if (!aligned(a->state, 16) || !aligned(a->codes, 16) || !aligned(a->scales, 16) ||
      !aligned(a->slots, 4) || !aligned(a->snaps, 4) || !aligned(a->err, 4))
    return KDA_ERR_ALIGNMENT;
  int dev = 0;
  DeviceFacts df;
  if (!current_device(&dev, &df)) return KDA_ERR_DEVICE;
  Params p;
  p.heads = a->heads;
  p.num_slots = a->num_slots;
  p.num_snaps = a->num_snaps;
  p.slots = a->slots;
  p.snaps = a->snaps;
  p.state = reinterpret_cast<float4 *>(a->state);
  p.codes = a->codes;
  p.scales = a->scales;
  p.err = a->err;
  const int grid = a->count * a->heads * kParts, threads = kWarps * 32;
  if (save) {
    if (a->bits == 8)
      save_kernel<8><<<grid, threads, 0, stream>>>(p);
    else
      save_kernel<4><<<grid, threads, 0, stream>>>(p);
  } else {
    if (a->bits == 8)
      load_kernel<8><<<grid, threads, 0, stream>>>(p);
    else
      load_kernel<4><<<grid, threads, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

}  // namespace snap
}  // namespace kda

extern "C" int kda_snapshot_save(const kda_snapshot_args *args, void *stream) {
  return kda::snap::run(args, true, static_cast<cudaStream_t>(stream));
}

extern "C" int kda_snapshot_load(const kda_snapshot_args *args, void *stream) {
  return kda::snap::run(args, false, static_cast<cudaStream_t>(stream));
}
