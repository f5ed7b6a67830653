// Shared by the operators on BF16 rows (convolution, scan, product): vectors of 8
// channels, softplus, and which sequence a piece of ragged rows belongs to.
#pragma once
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"

namespace kda {
namespace rows {

// The kernels here may start while the one before them in the stream ends
// (launch_following): each thread calls this before its first access to global memory.
// The kernel behind may start from then on, and so not before the one ahead is complete:
// what is two launches ahead is complete for a kernel that reads before its own wait.
__device__ __forceinline__ void follow() {
  griddep_wait();
  griddep_launch_dependents();
}

// 8 BF16 values of a 16-byte vector.
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

constexpr float kLog2e = 1.4426950408889634f;

// The same in pairs, for operations on two.
__device__ __forceinline__ f32x2 two(float v) { return pair(v, v); }
__device__ __forceinline__ f32x2 unpack2(uint32_t u) {
  return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ void pairs8(const uint4 &u, f32x2 (&f)[4]) {
  f[0] = unpack2(u.x), f[1] = unpack2(u.y), f[2] = unpack2(u.z), f[3] = unpack2(u.w);
}

// silu() of two values.  The bits of silu_approx, whose division is this product for
// all arguments from -87 on (all of FP32's compared); below, where both are under 2^-118,
// 0 for some of what it leaves.
__device__ __forceinline__ f32x2 silu2(f32x2 z) {
  float lo, hi;
  unpair(mul2(z, two(-kLog2e)), lo, hi);
  unpair(add2(pair(exp2_approx(lo), exp2_approx(hi)), two(1.0f)), lo, hi);
  return mul2(z, pair(rcp_approx(lo), rcp_approx(hi)));
}

// exp(x) for x <= 0, off by the approximate exp2 alone: the argument's rounding
// goes in as a factor.
__device__ __forceinline__ float exp_of(float x) {
  const float t = x * kLog2e;
  const float left = __fmaf_rn(x, 1.925963033e-8f, __fmaf_rn(x, kLog2e, -t));
  const float e = exp2_approx(t);
  return __fmaf_rn(e, left * 0.6931471806f, e);
}

// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|), to FP32's rounding also
// where it is small: log1p(e) = 2 atanh(q), q = e / (2 + e) <= 1/3, atanh(q) / q
// interpolated in q^2 at the Chebyshev points (degree 4, 4e-9).  NaN stays NaN.
__device__ __forceinline__ float softplus(float x) {
  const float e = exp_of(fabsf(x) > 100.0f ? -100.0f : -fabsf(x));     // (0 from -88 on)
  const float q = e * rcp_approx(2.0f + e);
  const float u = q * q;
  float t = 0.14078890f;
  t = __fmaf_rn(t, u, 0.13982579f);
  t = __fmaf_rn(t, u, 0.20012298f);
  t = __fmaf_rn(t, u, 0.33333161f);
  t = __fmaf_rn(t, u, 1.0f);
  const float l = 2.0f * q * t;
  return x > 0.0f ? x + l : l;
}

// The sequences of a prompt call.
struct Seqs {
  int count, tokens, longest, num_slots;
  const int32_t *starts, *src_slots, *dst_slots;
};

// One sequence: its rows and slots (0: none).
struct Seq {
  int start, len, src, dst;
};

// Resolves sequence b.  Returns the KDA_DEVERR_* flags it raises; a flagged
// sequence is skipped.
__device__ __forceinline__ int resolve(const Seqs &p, int b, Seq *s) {
  const int lo = __ldg(p.starts + b), hi = __ldg(p.starts + b + 1);
  int bad = 0;
  if (lo < 0 || hi < lo || hi > p.tokens || hi - lo > p.longest) bad |= KDA_DEVERR_SEQ;
  const int src = p.src_slots ? __ldg(p.src_slots + b) : 0;
  const int dst = p.dst_slots ? __ldg(p.dst_slots + b) : 0;
  if (src >= p.num_slots && src > 0) bad |= KDA_DEVERR_SLOT;
  if (dst >= p.num_slots && dst > 0) bad |= KDA_DEVERR_SLOT;
  s->start = lo;
  s->len = hi - lo;
  s->src = src > 0 ? src : 0;
  s->dst = dst > 0 ? dst : 0;
  return bad;
}

// Pieces of `piece` rows: sequence b's begin at number starts[b] / piece + b, so
// there are tokens / piece + count numbers and none is taken twice, however the
// lengths are spread.  Returns the sequence that number n falls to, by parts of an eighth
// whose starts are read together, as a call of few tokens is such waits (in range also
// where starts are out of order: what it finds is checked).
__device__ __forceinline__ int seq_of(const Seqs &p, int64_t n, int piece) {
  int lo = 0, hi = p.count;                 // first(lo) <= n < first(hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 7) / 8;
    int below = 0;                          // of the seven between, how many begin by n
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      const int64_t mid = lo + static_cast<int64_t>(k) * step;
      if (mid < hi && __ldg(p.starts + mid) / piece + mid <= n) ++below;
    }
    lo += below * step;
    if (hi - lo > step) hi = lo + step;
  }
  return lo;
}

inline int64_t pieces_of(int64_t tokens, int64_t seqs, int piece) { return tokens / piece + seqs; }

// Sizes that leave room to be rounded up to tiles in 32 bits.
constexpr int64_t kMostRows = 0x7fffff00ll;

inline bool aligned(const void *q, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(q) & (to - 1)) == 0;
}
// Row strides: multiples of 8 elements (16 bytes), no shorter than the row and
// short enough for a tensor map (2^40 bytes).
inline bool stride_ok(int64_t stride, int64_t width) {
  return stride % 8 == 0 && stride >= width && stride < (int64_t(1) << 38);
}

}  // namespace rows
}  // namespace kda
