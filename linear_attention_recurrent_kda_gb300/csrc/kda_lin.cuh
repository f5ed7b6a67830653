// Shared by the linear-attention kernels (one decay per head): the prompt
// call's parameters, the resolution of one sequence, and the slice of a state
// page that a warp keeps in registers in the recurrent forms.
//
// Per head, page S [value row i][key j] in FP32:
//   S_t = exp(g_t) S_{t-1} + v_t k_t^T,   o_t = scale * S_t q_t.
#pragma once
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"

namespace kda {
namespace lin {

constexpr int kDim = 128;                 // keys and value rows of a page
constexpr int kPage = kDim * kDim;        // floats of a page
constexpr int kRows = 8;                  // value rows a warp holds (recurrent forms)
constexpr int kSpan = 32 / kRows;         // lanes that share a row's sum

struct PromptParams {
  int seqs, heads, group, tokens, max_seq, num_slots, decay_rows;  // group = heads / qk_heads
  int slots, seg_len;     // sequences longer than seg_len are split; slots for their segments
  int64_t q_stride, k_stride, v_stride, o_stride;
  const __nv_bfloat16 *q, *k, *v;
  const float *decay;
  const int32_t *seq_starts, *src_slots, *dst_slots;
  float *state;
  __nv_bfloat16 *output;
  float scale;
  int32_t *err;
  float *ws_state;        // pages of the segments when slots > 0 (kda_lin_prompt.cu)
  float *ws_decay;        // their total decays
};

// One sequence of a prompt call: its rows and slots (0: none).
struct Seq {
  int start, len, src, dst;
};

// Resolves sequence b.  Returns the KDA_DEVERR_* flags it raises; a flagged
// sequence is skipped.
__device__ __forceinline__ int resolve_seq(const PromptParams &p, int b, Seq *s) {
  const int lo = __ldg(p.seq_starts + b), hi = __ldg(p.seq_starts + b + 1);
  int bad = 0;
  if (lo < 0 || hi < lo || hi > p.tokens || hi - lo > p.max_seq) bad |= KDA_DEVERR_SEQ;
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

__device__ __forceinline__ float *page_of(float *state, int slot, int heads, int h) {
  return state + (static_cast<int64_t>(slot) * heads + h) * kPage;
}

__device__ __forceinline__ void unpack4(const uint2 &u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xFFFF0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

// A token's decay exp(g) as keep + change, keep 0 or 1.  Rounded to FP32, a factor
// near 1 is off by up to 2^-25 the same way at every token: over the 12000 tokens
// of a slow head 1e-4 of the page.  exp(g) - 1 is off by 2^-25 of itself.
struct Decay {
  float keep, change;
};
__device__ __forceinline__ Decay decay_of(float g) {
  const float less = expm1f(g);
  const bool slow = less > -0.5f;
  return Decay{slow ? 1.0f : 0.0f, slow ? less : expf(g)};
}
// A chunk's or segment's decay 2^x as one factor, whose rounding would repeat in the
// same way: from 1/2 to 1 the part that FP32 cannot hold goes into the next one's factor
// (`carry`, 0 at first), so that the product over any number of them is off by 2^-24
// at most, at the cost of no second product for each element of the page (S + S (2^x - 1):
// 205 us instead of 195, 16 prompts x 64 heads).
__device__ __forceinline__ float carried_factor(float x, float &carry) {
  // (2^x - 1) / x on [-1, 0]: interpolated at the Chebyshev points, degree 5, off by
  // 2^-26 of it, with FP32's rounding 2^-22.9
  float t = 1.14919952e-4f;
  t = __fmaf_rn(t, x, 1.29163684e-3f);
  t = __fmaf_rn(t, x, 9.59703512e-3f);
  t = __fmaf_rn(t, x, 5.54992296e-2f);
  t = __fmaf_rn(t, x, 2.40226090e-1f);
  t = __fmaf_rn(t, x, 6.93147182e-1f);
  const float less = __fmaf_rn(t, x, carry);
  const float factor = 1.0f + less, left = less - (factor - 1.0f);      // exact
  const bool slow = fabsf(x + 0.5f) <= 0.5f;
  carry = slow ? left : 0.0f;
  return slow ? factor : exp2_approx(x);
}

// One token on a warp's kRows value rows: lane l holds keys 4l .. 4l+3 of each
// row.  vrow: lane r < kRows holds v of row r.  Returns S q of row lane / kSpan
// (FP32, unscaled).
__device__ __forceinline__ float token_step(float4 (&s)[kRows], const Decay &d, const float (&k)[4],
                                            const float (&q)[4], float vrow, int lane) {
  float dot[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float v = __shfl_sync(0xffffffffu, vrow, r);
    s[r].x = __fmaf_rn(s[r].x, d.keep, __fmaf_rn(s[r].x, d.change, v * k[0]));
    s[r].y = __fmaf_rn(s[r].y, d.keep, __fmaf_rn(s[r].y, d.change, v * k[1]));
    s[r].z = __fmaf_rn(s[r].z, d.keep, __fmaf_rn(s[r].z, d.change, v * k[2]));
    s[r].w = __fmaf_rn(s[r].w, d.keep, __fmaf_rn(s[r].w, d.change, v * k[3]));
    dot[r] = __fmaf_rn(s[r].w, q[3],
                       __fmaf_rn(s[r].z, q[2], __fmaf_rn(s[r].y, q[1], s[r].x * q[0])));
  }
  return warp_reduce_scatter<kRows>(dot, lane);
}

constexpr int kList = 8;       // units of a CTA that its kernel keeps in order and searches for

// Slots of the chunked form's segments, and its pages of workspace.
inline int64_t slots_of(int64_t tokens, int64_t seg_len) { return tokens / seg_len + 1; }
inline int64_t ws_pages(int64_t tokens, int64_t seg_len, int64_t heads) {
  return 2 * slots_of(tokens, seg_len) * heads;
}

// threads of a CTA and CTAs of a page in the segments' scan
constexpr int kSegmentThreads = 256, kSegmentBlocks = kPage / (4 * kSegmentThreads);

// The chunked form (kda_lin_prompt.cu): enqueues its kernels for checked
// parameters.  Returns a KDA_* code.
int launch_chunked(const PromptParams &p, int qk_heads, int dev, int sms, cudaStream_t stream);

}  // namespace lin
}  // namespace kda
