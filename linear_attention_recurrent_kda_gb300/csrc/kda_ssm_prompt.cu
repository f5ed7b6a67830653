// Selective scan over ragged prompts.
//
// A thread holds 16 states of a channel in registers (N / 16 lanes a channel) and
// walks the tokens; a CTA of 128 threads takes 2048 / N channels of one group.
// Tiles of 16 tokens of x, dt and z come by asynchronous copies, two tiles in
// flight; b and c go through registers into FP32 in shared memory, from where
// every lane of a warp reads the same words.
//
// Decays.  exp(s a) = ex2(s (a log2 e)) per token and state on the approximate exp2,
// and FP32 holds a factor near 1 to 2^-25: a state that remembers 1000 tokens would
// drift by 2e-5 of itself or more, to one side.  So over a tile the product of the
// factors that were used is kept too, less 1 (m <- m e + (e - 1), where e - 1 is exact),
// and at its end the state is corrected by (exp(a sum s) - 1 - m) h_0, with exp - 1 from
// a polynomial (decay_of): two operations per token and state and 20 per tile and
// state, where a polynomial at every token would take 8.
//
// Split sequences.  A sequence much longer than an SM's share is cut into pieces:
// scan_kernel<N, false> sums each piece's own contribution to the state (from zeros)
// and its steps; scan_kernel<N, true> runs the pieces side by side, each from the
// state that it sums up itself from the pieces before.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_ssm.cuh"

namespace kda {
namespace ssm {

constexpr int kThreads = 128;
constexpr int kTile = 16;                        // tokens
constexpr int kHeld = 16;                        // states of a thread

template <int kStates>
struct Stage {
  static constexpr int kLanes = kStates / kHeld;             // of a channel
  static constexpr int kChannels = kThreads / kLanes;        // of a CTA
  static constexpr int kVectors = kChannels / 8;             // 16 bytes each, of a row
  static constexpr int kShared = kTile * 2 * kStates / 8;    // vectors of b and c
  __nv_bfloat16 x[2][kTile][kChannels], dt[2][kTile][kChannels], z[2][kTile][kChannels];
  float b[2][kTile][kStates], c[2][kTile][kStates];
};

__device__ __forceinline__ void copy16(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
}

// The piece's start: the sequence's first state, and over the pieces before it,
// h <- exp(a s) h + u with their steps' sums s and contributions u.
template <int kStates>
__device__ __forceinline__ void start_of(const Params &p, const Seq &seq, int64_t first, int before,
                                         int channel, int held, const f32x2 (&a)[kHeld / 2],
                                         f32x2 (&h)[kHeld / 2]) {
#pragma unroll
  for (int i = 0; i < kHeld / 2; ++i) h[i] = 0;
  if (seq.src) {
    const float4 *from = reinterpret_cast<const float4 *>(state_of(p, seq.src, channel, kStates) + held);
#pragma unroll
    for (int i = 0; i < kHeld / 4; ++i) {
      const float4 v = from[i];
      h[2 * i] = pair(v.x, v.y);
      h[2 * i + 1] = pair(v.z, v.w);
    }
  }
  for (int j = 0; j < before; ++j) {
    const float s = p.ws_step[(first + j) * p.channels + channel];
    const float4 *u = reinterpret_cast<const float4 *>(
        p.ws_state + ((first + j) * p.channels + channel) * kStates + held);
#pragma unroll
    for (int i = 0; i < kHeld / 4; ++i) {
      const float4 v = u[i];
      float lo, hi, al, ah;
      unpair(h[2 * i], lo, hi);
      unpair(a[2 * i], al, ah);
      h[2 * i] = pair(decayed(lo, decay_of(s * al), v.x), decayed(hi, decay_of(s * ah), v.y));
      unpair(h[2 * i + 1], lo, hi);
      unpair(a[2 * i + 1], al, ah);
      h[2 * i + 1] = pair(decayed(lo, decay_of(s * al), v.z), decayed(hi, decay_of(s * ah), v.w));
    }
  }
}

// h + h_0 (exp(a s) - 1 - used) for decays down to 1/2 a tile; what a stronger one is
// off by, the next tiles forget.
__device__ __forceinline__ f32x2 corrected(f32x2 h, f32x2 h0, f32x2 a, float s, f32x2 product) {
  float v[2], v0[2], x[2], used[2];
  unpair(h, v[0], v[1]);
  unpair(h0, v0[0], v0[1]);
  unpair(a, x[0], x[1]);
  unpair(product, used[0], used[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Decay d = decay_of(s * x[i]);
    if (d.keep != 0.0f) v[i] = __fmaf_rn(v0[i], d.change - used[i], v[i]);
  }
  return pair(v[0], v[1]);
}

template <int kStates, bool kOut>
__global__ void __launch_bounds__(kThreads, 4) scan_kernel(const __grid_constant__ Params p) {
  using S = Stage<kStates>;
  extern __shared__ __align__(16) uint8_t raw[];
  S &st = *reinterpret_cast<S *>(raw);
  const int block = blockIdx.x % p.blocks;
  const int64_t n = blockIdx.x / p.blocks;
  const int group = block / p.group_blocks;
  const int channel0 = group * p.span + (block - group * p.group_blocks) * S::kChannels;
  const int wide = min(S::kChannels, (group + 1) * p.span - channel0);   // channels, 8 at least
  const int tid = threadIdx.x, mine = tid / S::kLanes, held = tid % S::kLanes * kHeld;
  Seq seq;
  int64_t first = 0;
  int piece = 0, rows, b;
  if (p.piece > 0) {
    if (kOut && block == 0 && tid == 0 && n < p.seqs.count && p.err) {   // each sequence's flags, once
      if (const int bad = resolve(p.seqs, static_cast<int>(n), &seq)) atomicOr(p.err, bad);
    }
    b = seq_of(p.seqs, n, p.piece);
    if (resolve(p.seqs, b, &seq)) return;
    first = seq.start / p.piece + b;
    const int64_t at = n - first;
    if (at < 0 || (at > 0 && at * p.piece >= seq.len)) return;
    piece = static_cast<int>(at);
    const int left = seq.len - piece * p.piece;
    if (!kOut && left <= p.piece) return;          // the last one's contribution goes nowhere
    rows = min(left, p.piece);
  } else {
    b = static_cast<int>(n);
    if (const int bad = resolve(p.seqs, b, &seq)) {
      if (p.err && block == 0 && tid == 0) atomicOr(p.err, bad);
      return;
    }
    rows = seq.len;
  }
  const int64_t row0 = seq.start + static_cast<int64_t>(piece) * p.piece;
  const bool live = mine < wide;
  const int channel = channel0 + (live ? mine : 0);

  auto load = [&](int tile) {                      // x, dt, z of a tile
    const int buf = tile & 1;
    for (int i = tid; i < kTile * S::kVectors; i += kThreads) {
      const int t = i / S::kVectors, v = i % S::kVectors;
      if (tile * kTile + t < rows && 8 * v < wide) {
        const int64_t row = row0 + tile * kTile + t;
        copy16(&st.x[buf][t][8 * v], p.x + row * p.x_stride + channel0 + 8 * v);
        copy16(&st.dt[buf][t][8 * v], p.dt + row * p.dt_stride + channel0 + 8 * v);
        if (kOut && p.z) copy16(&st.z[buf][t][8 * v], p.z + row * p.z_stride + channel0 + 8 * v);
      }
    }
  };
  constexpr int kMine = (S::kShared + kThreads - 1) / kThreads;
  uint4 shared[kMine];                             // this thread's part of b and c
  auto fetch = [&](int tile) {
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = tid + k * kThreads, t = i / (kStates / 4), v = i % (kStates / 4);
      shared[k] = make_uint4(0, 0, 0, 0);
      if (i < S::kShared && tile * kTile + t < rows) {
        const int64_t row = row0 + tile * kTile + t;
        shared[k] = __ldg(reinterpret_cast<const uint4 *>(
            (v < kStates / 8 ? p.b + row * p.b_stride : p.c + row * p.c_stride) + group * kStates) +
            v % (kStates / 8));
      }
    }
  };
  auto spread = [&](int tile) {
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = tid + k * kThreads, t = i / (kStates / 4), v = i % (kStates / 4);
      if (i < S::kShared) {
        float f[8];
        unpack8(shared[k], f);
        float4 *to = reinterpret_cast<float4 *>(
            (v < kStates / 8 ? st.b[tile & 1][t] : st.c[tile & 1][t]) + v % (kStates / 8) * 8);
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  };

  load(0);
  fetch(0);
  f32x2 a[kHeld / 2], h[kHeld / 2];
  {
    const float4 *from =
        reinterpret_cast<const float4 *>(p.a + static_cast<int64_t>(channel) * kStates + held);
#pragma unroll
    for (int i = 0; i < kHeld / 4; ++i) {
      const float4 v = __ldg(from + i);
      a[2 * i] = pair(v.x * kLog2e, v.y * kLog2e);
      a[2 * i + 1] = pair(v.z * kLog2e, v.w * kLog2e);
    }
  }
  const float skip = p.d ? __ldg(p.d + channel) : 0.0f;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + channel) : 0.0f;
  if (kOut) {
    start_of<kStates>(p, seq, first, piece, channel, held, a, h);
  } else {
#pragma unroll
    for (int i = 0; i < kHeld / 2; ++i) h[i] = 0;
  }
  float steps = 0.0f;                              // of the piece
  __nv_bfloat16 *out = kOut ? p.output + row0 * p.o_stride + channel : nullptr;

  for (int tile = 0; tile * kTile < rows; ++tile) {
    const int buf = tile & 1, count = min(kTile, rows - tile * kTile);
    copies_done();
    spread(tile);
    __syncthreads();
    if ((tile + 1) * kTile < rows) {
      load(tile + 1);
      fetch(tile + 1);
    }
    f32x2 h0[kHeld / 2], used[kHeld / 2];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeld / 2; ++i) {
      h0[i] = h[i];
      used[i] = 0;
    }
#pragma unroll 2
    for (int t = 0; t < count; ++t) {
      const float x = __bfloat162float(st.x[buf][t][mine]);
      float s = __bfloat162float(st.dt[buf][t][mine]) + bias;
      if (p.softplus) s = softplus(s);
      sum += s;
      const f32x2 ss = pair(s, s), sx = pair(s * x, s * x);
      const ulonglong2 *bn = reinterpret_cast<const ulonglong2 *>(st.b[buf][t] + held);
      const ulonglong2 *cn = reinterpret_cast<const ulonglong2 *>(st.c[buf][t] + held);
      f32x2 y = 0;
#pragma unroll
      for (int i = 0; i < kHeld / 2; i += 2) {
        const ulonglong2 bb = bn[i / 2];
        f32x2 e[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float lo, hi;
          unpair(mul2(ss, a[i + k]), lo, hi);
          e[k] = pair(exp2_approx(lo), exp2_approx(hi));
          used[i + k] = fma2(used[i + k], e[k], add2(e[k], pair(-1.0f, -1.0f)));
        }
        h[i] = fma2(h[i], e[0], mul2(sx, bb.x));
        h[i + 1] = fma2(h[i + 1], e[1], mul2(sx, bb.y));
        if (kOut) {
          const ulonglong2 cc = cn[i / 2];
          y = fma2(h[i], cc.x, y);
          y = fma2(h[i + 1], cc.y, y);
        }
      }
      if (kOut) {
        float lo, hi;
        unpair(y, lo, hi);
        float v = lo + hi;
#pragma unroll
        for (int o = 1; o < S::kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        v = __fmaf_rn(skip, x, v);
        if (p.z) v *= silu_approx(__bfloat162float(st.z[buf][t][mine]));
        if (live && held == 0) *out = __float2bfloat16_rn(v);
        out += p.o_stride;
      }
    }
    steps += sum;
#pragma unroll
    for (int i = 0; i < kHeld / 2; ++i) h[i] = corrected(h[i], h0[i], a[i], sum, used[i]);
  }
  if (!live) return;
  float *to = nullptr;
  if (!kOut) {
    to = p.ws_state + (n * p.channels + channel) * kStates + held;
    if (held == 0) p.ws_step[n * p.channels + channel] = steps;
  } else if (seq.dst && row0 + rows == seq.start + seq.len) {
    to = state_of(p, seq.dst, channel, kStates) + held;
  }
  if (to) {
#pragma unroll
    for (int i = 0; i < kHeld / 4; ++i) {
      float4 v;
      unpair(h[2 * i], v.x, v.y);
      unpair(h[2 * i + 1], v.z, v.w);
      reinterpret_cast<float4 *>(to)[i] = v;
    }
  }
}

template <int kStates>
static int launch(Params &p, cudaStream_t stream, int dev) {
  using S = Stage<kStates>;
  p.group_blocks = (p.span + S::kChannels - 1) / S::kChannels;
  p.blocks = p.channels / p.span * p.group_blocks;
  const int64_t units = p.piece > 0 ? pieces_of(p.seqs.tokens, p.seqs.count, p.piece) : p.seqs.count;
  if (units * p.blocks > 0x7fffffffll) return KDA_ERR_SHAPE;
  static std::atomic<bool> out_done[kMaxDevices], sum_done[kMaxDevices];
  if (!set_smem_limit_once(out_done, dev, reinterpret_cast<const void *>(scan_kernel<kStates, true>),
                           sizeof(S)) ||
      !set_smem_limit_once(sum_done, dev, reinterpret_cast<const void *>(scan_kernel<kStates, false>),
                           sizeof(S)))
    return KDA_ERR_LAUNCH;
  const int grid = static_cast<int>(units * p.blocks);
  if (p.piece > 0) {
    scan_kernel<kStates, false><<<grid, kThreads, sizeof(S), stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH;
  }
  scan_kernel<kStates, true><<<grid, kThreads, sizeof(S), stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

int launch_prompt(Params &p, int states, int dev, cudaStream_t stream) {
  return states == 16 ? launch<16>(p, stream, dev)
                      : states == 32 ? launch<32>(p, stream, dev) : launch<64>(p, stream, dev);
}

}  // namespace ssm
}  // namespace kda
