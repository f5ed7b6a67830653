// Selective scan: the single-token step, and the checks and dispatch of both
// calls.
//
// The step moves 8 bytes a state and has some 10 operations for it, 16 states a channel:
// it is near both bounds.  256 requests x 8192 channels x 16, 32 of them padding: 49 us,
// 5.1 TB/s (0.75 of the copy's rate), 67% of the issue slots taken.  Steps, gates and
// outputs by every lane of a channel for itself 75.7 us, a polynomial for each state by
// itself 55.3; 8 requests a thread 64 (134 registers), 64 or 256 threads a CTA 50 and 51,
// requests along a second grid dimension 50.7, 8 to 32 requests one after another in a CTA
// 52 to 56, 10 CTAs an SM in fewer registers 57.  4 x 1024: 3.0 us, a launch
// (4.1, and 51 for the large one, where it does not start while the kernel before ends).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <cmath>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_ssm.cuh"

namespace kda {
namespace ssm {

constexpr int kThreads = 128;
constexpr int kRequests = 4;     // of a thread: they share its part of a

// h <- 2^x h + add, two states: where the decay is near 1 (down to 2^-1/4) as
// h + h (2^x - 1) + add, for the reason at decayed; 2^x - 1 there is x times a
// polynomial (interpolated at the Chebyshev points, degree 3, off by 2^-24 of itself).  An
// infinite state stays (its parts would cancel to NaN), for 1% of the large step's time in
// as many registers (70 without a bound of them: 52.3 us).
__device__ __forceinline__ f32x2 decayed2(f32x2 h, f32x2 x, f32x2 add) {
  f32x2 t = fma2(two(8.977169171e-03f), x, two(5.540518463e-02f));
  t = fma2(t, x, two(2.402215898e-01f));
  t = mul2(fma2(t, x, two(6.931471229e-01f)), x);
  float lo, hi, tl, th, hl, hh;
  unpair(x, lo, hi);
  unpair(t, tl, th);
  unpair(h, hl, hh);
  const bool sl = fabsf(lo + 0.125f) <= 0.125f && fabsf(hl) < INFINITY;
  const bool sh = fabsf(hi + 0.125f) <= 0.125f && fabsf(hh) < INFINITY;
  const f32x2 change = pair(sl ? tl : exp2_approx(lo), sh ? th : exp2_approx(hi));
  const f32x2 keep = pair(sl ? hl : 0.0f, sh ? hh : 0.0f);
  return add2(keep, fma2(h, change, add));
}

// A thread: 4 states of a channel, of kRequests requests, all loads in flight at
// once.  What is the same for all states of a channel (the step, the gate, the output) is
// one lane's for each request.  Groups of channels are multiples of 8, so a warp's
// channels are of one group, and all there or none.
template <int kStates>
__global__ void __launch_bounds__(kThreads, 8) step_kernel(const __grid_constant__ Params p,
                                                           int blocks) {
  constexpr int kLanes = kStates / 4;
  follow();
  const int block = blockIdx.x % blocks, first = blockIdx.x / blocks * kRequests;
  const int channel = (block * kThreads + threadIdx.x) / kLanes, quad = threadIdx.x % kLanes;
  if (channel >= p.channels) return;
  int slot[kRequests];
#pragma unroll
  for (int i = 0; i < kRequests; ++i) slot[i] = first + i < p.batch ? __ldg(p.slots + first + i) : 0;
  // this lane's request
  const int mine = quad % kRequests, row = min(first + mine, p.batch - 1);
  const __nv_bfloat16 x_in = p.x[row * p.x_stride + channel];
  const __nv_bfloat16 dt_in = p.dt[row * p.dt_stride + channel];
  const __nv_bfloat16 z_in = p.z ? p.z[row * p.z_stride + channel] : __nv_bfloat16();
  const int states = channel / p.span * kStates + 4 * quad;
  uint2 b_in[kRequests], c_in[kRequests];
#pragma unroll
  for (int i = 0; i < kRequests; ++i) {
    const int64_t r = min(first + i, p.batch - 1);
    b_in[i] = __ldg(reinterpret_cast<const uint2 *>(p.b + r * p.b_stride + states));
    c_in[i] = __ldg(reinterpret_cast<const uint2 *>(p.c + r * p.c_stride + states));
  }
  float4 a = __ldg(reinterpret_cast<const float4 *>(p.a + static_cast<int64_t>(channel) * kStates) + quad);
  const float skip = p.d ? __ldg(p.d + channel) : 0.0f;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + channel) : 0.0f;
  ulonglong2 h[kRequests];
  const int64_t page = static_cast<int64_t>(p.channels) * kStates;       // floats of a slot
  float *const pool = p.state + static_cast<int64_t>(channel) * kStates + 4 * quad;
#pragma unroll
  for (int i = 0; i < kRequests; ++i) {
    if (slot[i] >= p.seqs.num_slots) {
      if (p.err && block == 0 && threadIdx.x == 0) atomicOr(p.err, KDA_DEVERR_SLOT);
      slot[i] = 0;
    }
    h[i] = make_ulonglong2(0, 0);
    if (slot[i] > 0) h[i] = __ldcs(reinterpret_cast<const ulonglong2 *>(pool + slot[i] * page));
  }
  const f32x2 a01 = pair(a.x * kLog2e, a.y * kLog2e), a23 = pair(a.z * kLog2e, a.w * kLog2e);
  const float x = __bfloat162float(x_in);
  float s = __bfloat162float(dt_in) + bias;
  if (p.softplus) s = softplus(s);
  const float sx = s * x;
  float y[kRequests];
#pragma unroll
  for (int i = 0; i < kRequests; ++i) {
    const f32x2 si = two(__shfl_sync(0xffffffffu, s, i, kRequests));
    const f32x2 sxi = two(__shfl_sync(0xffffffffu, sx, i, kRequests));
    h[i].x = decayed2(h[i].x, mul2(si, a01), mul2(sxi, unpack2(b_in[i].x)));
    h[i].y = decayed2(h[i].y, mul2(si, a23), mul2(sxi, unpack2(b_in[i].y)));
    if (slot[i] > 0) __stcs(reinterpret_cast<ulonglong2 *>(pool + slot[i] * page), h[i]);
    float lo, hi;
    unpair(fma2(unpack2(c_in[i].y), h[i].y, mul2(unpack2(c_in[i].x), h[i].x)), lo, hi);
    y[i] = lo + hi;
  }
#pragma unroll
  for (int o = kLanes / 2; o >= kRequests; o >>= 1)
#pragma unroll
    for (int i = 0; i < kRequests; ++i) y[i] += __shfl_xor_sync(0xffffffffu, y[i], o);
  // request `mine`'s sum over four lanes
  const bool high = quad & 2, odd = quad & 1;
  float keep[2] = {high ? y[2] : y[0], high ? y[3] : y[1]};
  const float send[2] = {high ? y[0] : y[2], high ? y[1] : y[3]};
  keep[0] += __shfl_xor_sync(0xffffffffu, send[0], 2);
  keep[1] += __shfl_xor_sync(0xffffffffu, send[1], 2);
  float sum = odd ? keep[1] : keep[0];
  sum += __shfl_xor_sync(0xffffffffu, odd ? keep[0] : keep[1], 1);
  sum = __fmaf_rn(skip, x, sum);
  if (p.z) sum *= silu_approx(__bfloat162float(z_in));
  int at = slot[0];
#pragma unroll
  for (int i = 1; i < kRequests; ++i) at = mine == i ? slot[i] : at;
  if (quad < kRequests && first + mine < p.batch)
    p.output[row * p.o_stride + channel] = __float2bfloat16_rn(at > 0 ? sum : 0.0f);
}

template <int kStates>
static int launch_step(const Params &p, cudaStream_t stream) {
  const int per = kThreads / (kStates / 4), blocks = (p.channels + per - 1) / per;
  const int64_t grid = (static_cast<int64_t>(p.batch) + kRequests - 1) / kRequests * blocks;
  if (grid > 0x7fffffffll) return KDA_ERR_SHAPE;
  return launch_following(step_kernel<kStates>, grid, kThreads, 0, 0, stream, p, blocks) ? KDA_SUCCESS
                                                                                         : KDA_ERR_LAUNCH;
}

template <class Args>
static int check(const Args *a, int64_t rows) {
  if (a->channels < 0 || a->groups < 1 || a->channels % (8 * int64_t(a->groups)) != 0)
    return KDA_ERR_SHAPE;
  if (rows < 0 || rows > kMostRows || (a->states != 16 && a->states != 32 && a->states != 64)) return KDA_ERR_SHAPE;
  if (int64_t(a->channels) * a->states > kMostRows) return KDA_ERR_SHAPE;
  const int64_t shared = int64_t(a->groups) * a->states;
  if (!stride_ok(a->x_stride, a->channels) || !stride_ok(a->dt_stride, a->channels) ||
      !stride_ok(a->b_stride, shared) || !stride_ok(a->c_stride, shared) ||
      !stride_ok(a->o_stride, a->channels) || (a->z && !stride_ok(a->z_stride, a->channels)))
    return KDA_ERR_SHAPE;
  return KDA_SUCCESS;
}
template <class Args>
static bool rows_aligned(const Args *a) {
  return aligned(a->x, 16) && aligned(a->dt, 16) && aligned(a->b, 16) && aligned(a->c, 16) &&
         aligned(a->z, 16) && aligned(a->output, 16) && aligned(a->a, 16) && aligned(a->state, 16) &&
         aligned(a->d, 4) && aligned(a->dt_bias, 4) && aligned(a->err, 4);
}
template <class Args>
static Params params_of(const Args *a) {
  Params p = {};
  p.seqs.num_slots = a->num_slots;
  p.channels = a->channels;
  p.span = a->channels / a->groups;
  p.softplus = a->softplus != 0;
  p.x_stride = a->x_stride;
  p.dt_stride = a->dt_stride;
  p.b_stride = a->b_stride;
  p.c_stride = a->c_stride;
  p.z_stride = a->z_stride;
  p.o_stride = a->o_stride;
  p.x = static_cast<const __nv_bfloat16 *>(a->x);
  p.dt = static_cast<const __nv_bfloat16 *>(a->dt);
  p.b = static_cast<const __nv_bfloat16 *>(a->b);
  p.c = static_cast<const __nv_bfloat16 *>(a->c);
  p.z = static_cast<const __nv_bfloat16 *>(a->z);
  p.a = a->a;
  p.d = a->d;
  p.dt_bias = a->dt_bias;
  p.state = a->state;
  p.output = static_cast<__nv_bfloat16 *>(a->output);
  p.err = a->err;
  return p;
}

static int run_step(const kda_ssm_step_args *a, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  if (const int rc = check(a, a->batch)) return rc;
  if (a->num_slots < 1) return KDA_ERR_SHAPE;
  if (a->batch == 0 || a->channels == 0) return KDA_SUCCESS;
  if (!a->x || !a->dt || !a->a || !a->b || !a->c || !a->slots || !a->state || !a->output)
    return KDA_ERR_NULL_POINTER;
  if (!rows_aligned(a) || !aligned(a->slots, 4)) return KDA_ERR_ALIGNMENT;
  int dev = 0;
  DeviceFacts df;
  if (!current_device(&dev, &df)) return KDA_ERR_DEVICE;
  Params p = params_of(a);
  p.slots = a->slots;
  p.batch = a->batch;
  return a->states == 16 ? launch_step<16>(p, stream)
                         : a->states == 32 ? launch_step<32>(p, stream) : launch_step<64>(p, stream);
}

// How a prompt call runs.
struct Plan {
  int held, piece;         // states of a thread; rows of a piece (0: sequences stay whole)
  int64_t workspace;       // bytes
};
constexpr int kSms = 152, kCtas = 6;     // pieces: two for each of the 3 CTAs that an SM holds
constexpr int kShortestPiece = 256;      // rows

// Whether so many sequences or pieces are a grid that can be launched (CTAs are of one
// group's channels: kda_ssm_prompt.cu).
static bool launchable(const kda_ssm_prompt_args *a, int64_t units, int held) {
  const int64_t per = 128 / (a->states / held), span = a->channels / a->groups;
  return units * a->groups * ((span + per - 1) / per) <= 0x7fffffffll;
}

static int plan_prompt(const kda_ssm_prompt_args *a, Plan *plan) {
  if (const int rc = check(a, a->tokens)) return rc;
  const bool pool = a->src_slots || a->dst_slots;
  if (a->seqs < 0 || a->seqs > kMostRows || a->max_seq < 0 || (pool && a->num_slots < 1)) return KDA_ERR_SHAPE;
  if (a->path < 0 || a->path > 2) return KDA_ERR_PATH;
  const int64_t longest = a->max_seq < a->tokens ? a->max_seq : a->tokens;
  const int64_t threads = static_cast<int64_t>(a->channels) * (a->states / 16);
  const int64_t blocks = (threads + 127) / 128;          // CTAs of a sequence or piece
  // us.  A call takes as long as its longest sequence alone or as all the work, and a little
  // longer where the two are near.  8 states a thread are faster alone and slower in all (8
  // sequences, 9159 tokens x 4096 channels: 237 us with 8, 297 with 16 where the longest has
  // 2047, 249 and 231 where all have 1145).  Of 19 shapes, 10% more than the other's at most.
  const double work = static_cast<double>(a->tokens) * blocks;
  const double with8 = std::hypot(0.072 * longest, 0.78e-3 * work);
  const double with16 = std::hypot(0.125 * longest, 0.66e-3 * work);
  plan->held = with8 < with16 ? 8 : 16;
  plan->piece = 0;
  plan->workspace = 0;
  const int whole = launchable(a, a->seqs, plan->held) ? KDA_SUCCESS : KDA_ERR_SHAPE;
  if (a->path == 1 || blocks == 0 || longest <= kShortestPiece) return whole;
  // As many pieces as run at a time (each sequence's last one may be short); two passes over
  // all tokens, and each piece sums up those before it.  (One sequence of 2048 x 4096
  // channels 150 us whole, 92 in pieces; of 512 43 and 61; the 8 ragged ones 237 and 336.  All of 16 states;
  // with 32 and 64 the ragged ones take 389 and 1297 us, 8192 x 4096 485 and 1409.)
  int64_t pieces = kSms * kCtas / blocks - (a->seqs - 1);
  if (pieces < 1) pieces = 1;
  int64_t piece = (a->tokens / pieces + 16) / 16 * 16;
  if (piece < kShortestPiece || piece >= longest) piece = kShortestPiece;
  const double split = std::fmax(1.02e-3 * work, 0.23 * piece) + 1.3 * (longest / piece);
  if (a->path == 0 && (with8 < with16 ? with8 : with16) < split) return whole;
  const int64_t units = pieces_of(a->tokens, a->seqs, static_cast<int>(piece));
  if (!launchable(a, units, 16)) return a->path == 0 ? whole : KDA_ERR_SHAPE;
  plan->held = 16;
  plan->piece = static_cast<int>(piece);
  plan->workspace = units * a->channels * (a->states + 1) * 4;
  return KDA_SUCCESS;
}

static int run_prompt(const kda_ssm_prompt_args *a, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  Plan plan;
  if (const int rc = plan_prompt(a, &plan)) return rc;
  if (a->seqs == 0 || a->channels == 0) return KDA_SUCCESS;
  if (!a->seq_starts || !a->a || ((a->src_slots || a->dst_slots) && !a->state)) return KDA_ERR_NULL_POINTER;
  if (a->tokens > 0 && (!a->x || !a->dt || !a->b || !a->c || !a->output))
    return KDA_ERR_NULL_POINTER;
  if (!rows_aligned(a) || !aligned(a->seq_starts, 4) || !aligned(a->src_slots, 4) ||
      !aligned(a->dst_slots, 4))
    return KDA_ERR_ALIGNMENT;
  if (plan.workspace > 0 && (!a->workspace || !aligned(a->workspace, 256) ||
                             a->workspace_bytes < plan.workspace))
    return KDA_ERR_WORKSPACE;
  int dev = 0;
  DeviceFacts df;
  if (!current_device(&dev, &df)) return KDA_ERR_DEVICE;
  Params p = params_of(a);
  p.seqs.count = a->seqs;
  p.seqs.tokens = a->tokens;
  p.seqs.longest = a->max_seq < a->tokens ? a->max_seq : a->tokens;
  p.seqs.starts = a->seq_starts;
  p.seqs.src_slots = a->src_slots;
  p.seqs.dst_slots = a->dst_slots;
  p.piece = plan.piece;
  if (plan.piece > 0) {
    p.ws_state = static_cast<float *>(a->workspace);
    p.ws_step = p.ws_state + pieces_of(a->tokens, a->seqs, plan.piece) * a->channels * a->states;
  }
  return launch_prompt(p, a->states, plan.held, dev, stream);
}

}  // namespace ssm
}  // namespace kda

extern "C" int kda_ssm_step(const kda_ssm_step_args *args, void *stream) {
  return kda::ssm::run_step(args, static_cast<cudaStream_t>(stream));
}

extern "C" int kda_ssm_prompt(const kda_ssm_prompt_args *args, void *stream) {
  return kda::ssm::run_prompt(args, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t kda_ssm_prompt_workspace(const kda_ssm_prompt_args *args) {
  if (!args) return -1;
  kda::ssm::Plan plan;
  return kda::ssm::plan_prompt(args, &plan) ? 0 : plan.workspace;
}
