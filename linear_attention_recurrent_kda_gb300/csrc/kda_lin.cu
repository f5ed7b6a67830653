// Linear attention with one decay per head: the single-token step, the
// token-by-token prompt form, and the checks and dispatch of both calls.
//
// Both forms keep a page slice in registers: a warp holds 8 value rows, lane l
// the keys 4l .. 4l+3 of each (a row is one 512-byte access of the warp), so that
// S q needs one reduce-scatter for 8 rows.  A product v k is of two BF16 values
// and exact in FP32; the decay is applied as decay_of says.
//
// The step is HBM-bound (a page read and written per item, 128 KiB against
// 160 kflop).  CTAs of two warps, an eighth of a page each: all loads of a
// thread are in flight at once and the many small CTAs of an SM keep its
// memory queue full without a pipeline; a batch of few requests still spreads
// over the SMs.  GB300: 256 requests x 32 heads 159 us = 6.8 TB/s, the copy's
// rate (16 rows a warp: 160 us); 64 x 32 with 8 padded 38.6 us (0.90); 4 x 8 2.3 us,
// a launch.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_lin.cuh"

namespace kda {
namespace lin {

constexpr int kWarps = 2;                               // of a CTA (recurrent forms)
constexpr int kParts = kDim / (kWarps * kRows);         // CTAs of a page
constexpr int kMostHeads = 1 << 16;

struct StepParams {
  int heads, group, num_slots, decay_rows;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const __nv_bfloat16 *q, *k, *v;
  const float *decay;
  const int32_t *slots;
  float *state;
  __nv_bfloat16 *output;
  float scale;
  int32_t *err;
};

__global__ void __launch_bounds__(kWarps * 32) step_kernel(const __grid_constant__ StepParams p) {
  const int part = blockIdx.x % kParts, item = blockIdx.x / kParts;
  const int r = item / p.heads, h = item % p.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = (part * kWarps + warp) * kRows;
  __nv_bfloat16 *out = p.output + r * p.o_stride + h * kDim + row0;
  const int slot = __ldg(p.slots + r);
  if (slot <= 0 || slot >= p.num_slots) {
    if (lane < kRows) out[lane] = __float2bfloat16_rn(0.0f);
    if (slot >= p.num_slots && p.err && threadIdx.x == 0) atomicOr(p.err, KDA_DEVERR_SLOT);
    return;
  }
  float4 *page = reinterpret_cast<float4 *>(page_of(p.state, slot, p.heads, h) + row0 * kDim) + lane;
  float4 s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) s[i] = __ldcs(page + i * 32);
  float k[4], q[4];
  unpack4(__ldg(reinterpret_cast<const uint2 *>(p.k + r * p.k_stride + h / p.group * kDim) + lane), k);
  unpack4(__ldg(reinterpret_cast<const uint2 *>(p.q + r * p.q_stride + h / p.group * kDim) + lane), q);
  const float v = __bfloat162float(p.v[r * p.v_stride + h * kDim + row0 + (lane & (kRows - 1))]);
  const Decay d =
      decay_of(__ldg(p.decay + (p.decay_rows ? static_cast<int64_t>(r) * p.heads : 0) + h));
  const float o = token_step(s, d, k, q, v, lane);
#pragma unroll
  for (int i = 0; i < kRows; ++i) __stcs(page + i * 32, s[i]);
  if (lane % kSpan == 0) out[lane / kSpan] = __float2bfloat16_rn(p.scale * o);
}

// Token by token over a sequence: the operands of token t + 1 are loaded while
// token t is computed.
__global__ void __launch_bounds__(kWarps * 32)
    recurrent_kernel(const __grid_constant__ PromptParams p) {
  const int part = blockIdx.x % kParts, item = blockIdx.x / kParts;
  const int b = item / p.heads, h = item % p.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = (part * kWarps + warp) * kRows;
  Seq seq;
  if (const int bad = resolve_seq(p, b, &seq)) {
    if (p.err && threadIdx.x == 0) atomicOr(p.err, bad);
    return;
  }
  float4 s[kRows];
  if (seq.src) {
    const float4 *page =
        reinterpret_cast<const float4 *>(page_of(p.state, seq.src, p.heads, h) + row0 * kDim) + lane;
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = page[i * 32];
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  const uint2 *kp =
      reinterpret_cast<const uint2 *>(p.k + seq.start * p.k_stride + h / p.group * kDim) + lane;
  const uint2 *qp =
      reinterpret_cast<const uint2 *>(p.q + seq.start * p.q_stride + h / p.group * kDim) + lane;
  const __nv_bfloat16 *vp =
      p.v + seq.start * p.v_stride + h * kDim + row0 + (lane & (kRows - 1));
  const float *gp = p.decay + (p.decay_rows ? static_cast<int64_t>(seq.start) * p.heads : 0) + h;
  const int64_t g_step = p.decay_rows ? p.heads : 0;
  __nv_bfloat16 *out = p.output + seq.start * p.o_stride + h * kDim + row0 + lane / kSpan;
  uint2 kn = make_uint2(0, 0), qn = kn;
  __nv_bfloat16 vn = __float2bfloat16_rn(0.0f);
  float gn = 0.0f;
  for (int t = 0; t <= seq.len; ++t) {
    const uint2 kc = kn, qc = qn;
    const float v = __bfloat162float(vn);
    const Decay d = decay_of(gn);
    if (t < seq.len) {
      kn = __ldg(kp);
      qn = __ldg(qp);
      vn = *vp;
      gn = __ldg(gp);
      kp += p.k_stride / 4;
      qp += p.q_stride / 4;
      vp += p.v_stride;
      gp += g_step;
    }
    if (t == 0) continue;
    float k[4], q[4];
    unpack4(kc, k);
    unpack4(qc, q);
    const float o = token_step(s, d, k, q, v, lane);
    if (lane % kSpan == 0) *out = __float2bfloat16_rn(p.scale * o);
    out += p.o_stride;
  }
  if (seq.dst) {
    float4 *page =
        reinterpret_cast<float4 *>(page_of(p.state, seq.dst, p.heads, h) + row0 * kDim) + lane;
#pragma unroll
    for (int i = 0; i < kRows; ++i) __stcs(page + i * 32, s[i]);
  }
}

static bool aligned(const void *q, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(q) & (to - 1)) == 0;
}

// Row strides: multiples of 8 elements (16 bytes), no shorter than the row and
// short enough for a tensor map (2^40 bytes).
static bool stride_ok(int64_t stride, int64_t width) {
  return stride % 8 == 0 && stride >= width && stride < (int64_t(1) << 38);
}

template <class Args>
static int check_common(const Args *a, int64_t count) {
  if (count < 0 || a->heads < 0 || a->qk_heads < 1 || a->heads % a->qk_heads != 0)
    return KDA_ERR_SHAPE;
  if (a->decay_rows != 0 && a->decay_rows != 1) return KDA_ERR_SHAPE;
  if (a->heads > kMostHeads) return KDA_ERR_SHAPE;
  if (count * a->heads * kParts > 0x7fffffffll) return KDA_ERR_SHAPE;
  const int64_t kw = int64_t(a->qk_heads) * kDim, vw = int64_t(a->heads) * kDim;
  if (!stride_ok(a->q_stride, kw) || !stride_ok(a->k_stride, kw) || !stride_ok(a->v_stride, vw) ||
      !stride_ok(a->o_stride, vw))
    return KDA_ERR_SHAPE;
  return KDA_SUCCESS;
}

template <class Args>
static bool rows_aligned(const Args *a) {
  return aligned(a->q, 16) && aligned(a->k, 16) && aligned(a->v, 16) && aligned(a->output, 16) &&
         aligned(a->state, 16) && aligned(a->decay, 4) && aligned(a->err, 4);
}

static int run_step(const kda_lin_step_args *a, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  if (const int rc = check_common(a, a->batch)) return rc;
  if (a->num_slots < 1) return KDA_ERR_SHAPE;
  if (a->batch == 0 || a->heads == 0) return KDA_SUCCESS;
  if (!a->q || !a->k || !a->v || !a->decay || !a->slots || !a->state || !a->output)
    return KDA_ERR_NULL_POINTER;
  if (!rows_aligned(a) || !aligned(a->slots, 4)) return KDA_ERR_ALIGNMENT;
  int dev = 0;
  DeviceFacts df;
  if (!current_device(&dev, &df)) return KDA_ERR_DEVICE;
  StepParams p;
  p.heads = a->heads;
  p.group = a->heads / a->qk_heads;
  p.num_slots = a->num_slots;
  p.decay_rows = a->decay_rows;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.o_stride = a->o_stride;
  p.q = static_cast<const __nv_bfloat16 *>(a->q);
  p.k = static_cast<const __nv_bfloat16 *>(a->k);
  p.v = static_cast<const __nv_bfloat16 *>(a->v);
  p.decay = a->decay;
  p.slots = a->slots;
  p.state = a->state;
  p.output = static_cast<__nv_bfloat16 *>(a->output);
  p.scale = a->scale;
  p.err = a->err;
  step_kernel<<<a->batch * a->heads * kParts, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

// How a prompt call runs.
struct Plan {
  bool chunked;
  int slots, seg_len;     // of segments; 0 slots: sequences stay whole
  int64_t workspace;      // bytes
};

// Short sequences take the recurrent form, which reads each page once and starts
// at once.  12 tokens: 7.5 us against 7.7 chunked (32 items of 128 x 128), 11.1
// against 8.2 (128 items), 123 against 76 (2048 items); 8 tokens: 5.7 against 7.7,
// 8.4 against 8.2 and 91 against 76; 4 tokens: 4.0 against 7.7, 5.6 against 8.2 and 62
// against 75.
constexpr int kRecurrentMost = 6, kRecurrentMostFew = 12, kFewItems = 64;
constexpr int kShares = 152;            // SMs that the work is shared among
constexpr int kShortestSegment = 256;   // tokens
constexpr int kSplitCost = 896;         // of splitting, in tokens of one head

// The sizes' part of the checks, and the plan.
static int plan_prompt(const kda_lin_prompt_args *a, Plan *plan) {
  if (const int rc = check_common(a, a->seqs)) return rc;
  if (a->tokens < 0 || a->max_seq < 0 || (a->state && a->num_slots < 1)) return KDA_ERR_SHAPE;
  if (a->path < 0 || a->path > 2) return KDA_ERR_PATH;
  const int64_t longest = a->max_seq < a->tokens ? a->max_seq : a->tokens;
  const int64_t items = static_cast<int64_t>(a->seqs) * a->heads;
  const int recurrent_most = items <= kFewItems ? kRecurrentMostFew : kRecurrentMost;
  plan->chunked = longest > 0 && (a->path == 2 || (a->path == 0 && longest > recurrent_most));
  plan->slots = 0;
  plan->seg_len = longest > 0 ? static_cast<int>(longest) : 1;
  plan->workspace = 0;
  if (plan->chunked) {
    // A sequence much longer than an SM's share of all tokens x heads would keep
    // its SM busy alone.  Split, the share costs a second pass over keys and values
    // (0.6 of the first) and two more launches: it pays from 2 shares and 896 tokens
    // on (one sequence, whole and split: 1 head of 1024 tokens 26 and 26 us, of 768 21
    // and 26, of 2048 45 and 27; 8 heads of 1024 26 and 28, of 1280 31 and 28, of 8192
    // 165 and 46; 16 heads of 1024 26 and 28, of 1536 36 and 29; 32 heads of 1280 31
    // and 39, of 2048 46 and 45; 64 heads of 2048 52 and 70, of 4096 98 and 107).
    // Segments of a quarter share even out what the last ones leave.
    const int64_t share = static_cast<int64_t>(a->tokens) * a->heads / kShares;
    int64_t len = (share / 4 + 127) / 128 * 128;
    if (len < kShortestSegment) len = kShortestSegment;
    // (the slots of the segments are at most 4 an SM and one for each head; with
    // more heads than that leaves room for, there are enough units without)
    if (longest > 2 * share + kSplitCost && slots_of(a->tokens, len) * a->heads <= kList * kShares) {
      plan->seg_len = static_cast<int>(len);
      plan->slots = static_cast<int>(slots_of(a->tokens, len));
      if ((static_cast<int64_t>(plan->slots) + a->seqs) * a->heads > 0x7fffffffll)
        return KDA_ERR_SHAPE;
      plan->workspace = ws_pages(a->tokens, len, a->heads) * (kPage + 1) * 4;
    }
  }
  return KDA_SUCCESS;
}

static int run_prompt(const kda_lin_prompt_args *a, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  Plan plan;
  if (const int rc = plan_prompt(a, &plan)) return rc;
  if (a->seqs == 0 || a->heads == 0) return KDA_SUCCESS;
  if (!a->seq_starts) return KDA_ERR_NULL_POINTER;
  if (a->tokens > 0 && (!a->q || !a->k || !a->v || !a->decay || !a->output))
    return KDA_ERR_NULL_POINTER;
  if ((a->src_slots || a->dst_slots) && !a->state) return KDA_ERR_NULL_POINTER;
  if (!rows_aligned(a) || !aligned(a->seq_starts, 4) || !aligned(a->src_slots, 4) ||
      !aligned(a->dst_slots, 4))
    return KDA_ERR_ALIGNMENT;
  if (plan.workspace > 0 && (!a->workspace || !aligned(a->workspace, 256) ||
                             a->workspace_bytes < plan.workspace))
    return KDA_ERR_WORKSPACE;
  int dev = 0;
  DeviceFacts df;
  if (!current_device(&dev, &df)) return KDA_ERR_DEVICE;
  PromptParams p = {};
  p.seqs = a->seqs;
  p.heads = a->heads;
  p.group = a->heads / a->qk_heads;
  p.tokens = a->tokens;
  p.max_seq = a->max_seq < a->tokens ? a->max_seq : a->tokens;
  p.num_slots = a->num_slots;
  p.decay_rows = a->decay_rows;
  p.slots = plan.slots;
  p.seg_len = plan.seg_len;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.o_stride = a->o_stride;
  p.q = static_cast<const __nv_bfloat16 *>(a->q);
  p.k = static_cast<const __nv_bfloat16 *>(a->k);
  p.v = static_cast<const __nv_bfloat16 *>(a->v);
  p.decay = a->decay;
  p.seq_starts = a->seq_starts;
  p.src_slots = a->src_slots;
  p.dst_slots = a->dst_slots;
  p.state = a->state;
  p.output = static_cast<__nv_bfloat16 *>(a->output);
  p.scale = a->scale;
  p.err = a->err;
  if (plan.chunked) {
    if (plan.workspace > 0) {
      p.ws_state = static_cast<float *>(a->workspace);
      p.ws_decay = p.ws_state + ws_pages(p.tokens, p.seg_len, p.heads) * kPage;
    }
    return launch_chunked(p, a->qk_heads, dev, df.sms, stream);
  }
  recurrent_kernel<<<a->seqs * a->heads * kParts, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

}  // namespace lin
}  // namespace kda

extern "C" int kda_lin_step(const kda_lin_step_args *args, void *stream) {
  return kda::lin::run_step(args, static_cast<cudaStream_t>(stream));
}

extern "C" int kda_lin_prompt(const kda_lin_prompt_args *args, void *stream) {
  return kda::lin::run_prompt(args, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t kda_lin_prompt_workspace(const kda_lin_prompt_args *args) {
  if (!args) return -1;
  kda::lin::Plan plan;
  return kda::lin::plan_prompt(args, &plan) ? 0 : plan.workspace;
}
