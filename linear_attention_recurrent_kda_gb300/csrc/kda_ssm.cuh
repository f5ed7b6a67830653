// Shared by the selective scan's kernels: parameters, and the arithmetic of one
// token.  Per channel, with N states:
//   s = softplus(dt + dt_bias),  h_n <- exp(s a_n) h_n + s x b_n,
//   y = sum_n c_n h_n + d x,     out = y silu(z).
#pragma once
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <cmath>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_rows.cuh"

namespace kda {
namespace ssm {

using namespace rows;

struct Params {
  Seqs seqs;                     // prompt
  const int32_t *slots;          // step
  int batch;
  int channels, span, softplus;  // span: channels of a group
  int64_t x_stride, dt_stride, b_stride, c_stride, z_stride, o_stride;
  const __nv_bfloat16 *x, *dt, *b, *c, *z;
  const float *a, *d, *dt_bias;
  float *state;
  __nv_bfloat16 *output;
  int32_t *err;
  // prompt: CTAs across the channels, and of a group; with pieces (> 0 rows each), what
  // they leave: states [piece][channel][N] and sums of steps [piece][channel]
  int blocks, group_blocks, piece;
  float *ws_state, *ws_step;
};

// 2^x - 1 on [-1, 0]: x times a polynomial, interpolated at the Chebyshev points, degree 5,
// off by 2^-26 of itself.
__device__ __forceinline__ float less_one(float x) {
  float t = 1.14919952e-4f;
  t = __fmaf_rn(t, x, 1.29163684e-3f);
  t = __fmaf_rn(t, x, 9.59703512e-3f);
  t = __fmaf_rn(t, x, 5.54992296e-2f);
  t = __fmaf_rn(t, x, 2.40226090e-1f);
  t = __fmaf_rn(t, x, 6.93147182e-1f);
  return t * x;
}
// 2^x h + add; where the decay is down to 1/2 as h + h (2^x - 1) + add: near 1 a factor
// rounded to FP32 is off the same way at every token of a constant step, and a slow state
// drifts (2^-25 a token); 2^x - 1 is off by 2^-23 of itself, which no number of tokens
// adds up.  (Not so an infinite state, whose parts would cancel to NaN.)
__device__ __forceinline__ float decayed(float h, float x, float add) {
  const bool slow = fabsf(x + 0.5f) <= 0.5f && fabsf(h) < INFINITY;
  return (slow ? h : 0.0f) + __fmaf_rn(h, slow ? less_one(x) : exp2_approx(x), add);
}

// 4 BF16 values of an 8-byte vector.
__device__ __forceinline__ void unpack4(const uint2 &u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xFFFF0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

__device__ __forceinline__ float *state_of(const Params &p, int slot, int channel, int states) {
  return p.state + (static_cast<int64_t>(slot) * p.channels + channel) * states;
}

// Enqueues the prompt form for checked parameters, with `held` (8, or 16, as pieces
// need) states a thread.  Returns a KDA_* code.
int launch_prompt(Params &p, int states, int held, int dev, cudaStream_t stream);

}  // namespace ssm
}  // namespace kda
