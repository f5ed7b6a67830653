// Selective scan over ragged prompts.
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

// Token by token: a thread holds 4 states of a channel, kLanes = N / 4 lanes a
// channel.  (A warp's channels are all of one group, and all there or none: groups
// are multiples of 8 channels.)
template <int kStates>
__global__ void __launch_bounds__(kThreads) prompt_kernel(const __grid_constant__ Params p,
                                                          int blocks) {
  constexpr int kLanes = kStates / 4;
  const int block = blockIdx.x % blocks, b = blockIdx.x / blocks;
  const int channel = (block * kThreads + threadIdx.x) / kLanes, quad = threadIdx.x % kLanes;
  Seq seq;
  if (const int bad = resolve(p.seqs, b, &seq)) {
    if (p.err && block == 0 && threadIdx.x == 0) atomicOr(p.err, bad);
    return;
  }
  if (channel >= p.channels) return;
  float4 a = __ldg(reinterpret_cast<const float4 *>(p.a + static_cast<int64_t>(channel) * kStates) + quad);
  a.x *= kLog2e, a.y *= kLog2e, a.z *= kLog2e, a.w *= kLog2e;
  const float d = p.d ? __ldg(p.d + channel) : 0.0f;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + channel) : 0.0f;
  float4 h = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (seq.src) h = reinterpret_cast<const float4 *>(state_of(p, seq.src, channel, kStates))[quad];
  const int states = channel / p.span * kStates + 4 * quad;
  for (int t = 0; t < seq.len; ++t) {
    const int64_t row = seq.start + t;
    const float x = __bfloat162float(p.x[row * p.x_stride + channel]);
    float s = __bfloat162float(p.dt[row * p.dt_stride + channel]) + bias;
    if (p.softplus) s = softplus(s);
    float bn[4], cn[4];
    unpack4(__ldg(reinterpret_cast<const uint2 *>(p.b + row * p.b_stride + states)), bn);
    unpack4(__ldg(reinterpret_cast<const uint2 *>(p.c + row * p.c_stride + states)), cn);
    const float sx = s * x;
    h.x = decayed(h.x, decay_of(s * a.x), sx * bn[0]);
    h.y = decayed(h.y, decay_of(s * a.y), sx * bn[1]);
    h.z = decayed(h.z, decay_of(s * a.z), sx * bn[2]);
    h.w = decayed(h.w, decay_of(s * a.w), sx * bn[3]);
    float y = cn[0] * h.x + cn[1] * h.y + cn[2] * h.z + cn[3] * h.w;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (quad == 0) {
      y = __fmaf_rn(d, x, y);
      if (p.z) y *= silu_approx(__bfloat162float(p.z[row * p.z_stride + channel]));
      p.output[row * p.o_stride + channel] = __float2bfloat16_rn(y);
    }
  }
  if (seq.dst) reinterpret_cast<float4 *>(state_of(p, seq.dst, channel, kStates))[quad] = h;
}

template <int kStates>
static int launch(const Params &p, cudaStream_t stream) {
  const int per = kThreads / (kStates / 4), blocks = (p.channels + per - 1) / per;
  if (static_cast<int64_t>(blocks) * p.seqs.count > 0x7fffffffll) return KDA_ERR_SHAPE;
  prompt_kernel<kStates><<<blocks * p.seqs.count, kThreads, 0, stream>>>(p, blocks);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

int launch_prompt(const Params &p, int states, cudaStream_t stream) {
  return states == 16 ? launch<16>(p, stream)
                      : states == 32 ? launch<32>(p, stream) : launch<64>(p, stream);
}

}  // namespace ssm
}  // namespace kda
