// Short causal depthwise convolution with SiLU, over ragged prompts and for single
// tokens:  y_t = bias + sum_j w_j x_{t - taps + 1 + j}, per channel.
//
// HBM-bound: 4 bytes a token and channel against 2 * taps flop and one SiLU.  A
// thread holds 8 channels (one 16-byte vector of a row): their weights and the
// last inputs stay in registers while it walks a piece of a sequence, so every
// input is read once (and taps - 1 rows again per piece, from L2); the next four rows
// come while four are worked on.  The sum runs from the bias on, oldest input first,
// and the SiLU is the KDA step's, so a prompt leaves the step's own bits.
//
// GB300: 9159 tokens x 12288 channels 79 us, 5.7 TB/s (0.84 of the copy's rate); one
// channel to an operation and no rows ahead 113 us, weights and the first rows behind the
// windows 82 (4 x 9 tokens: 4.1 us, 3.7 so).  Not kept: pieces of 16 rows 91 us,
// of 64 82 (with half the threads for small calls), of 128 96; 2 rows ahead 99, 8 85; 4
// channels a thread 79-85 (before), and 16.8 instead of 12.3 us for the step of 256 requests x 8192
// channels (10.0 us, 5.1 TB/s, since it starts while the kernel before ends).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_rows.cuh"

namespace kda {
namespace conv {

using namespace rows;

constexpr int kThreads = 128;
constexpr int kPiece = 32;       // rows a thread walks
constexpr int kBatch = 4;        // of them in flight

struct Params {
  Seqs seqs;                     // prompt
  const int32_t *slots;          // step
  int batch;
  int64_t pieces;
  int vectors, channels, part, width, silu;    // part: channels of a block of weights
  int64_t x_stride, o_stride;
  const __nv_bfloat16 *x, *weight, *bias;
  void *window;
  __nv_bfloat16 *output;
  int32_t *err;
};

// 8 channels, two to an operation.
template <int kTaps>
struct Channels {
  f32x2 w[kTaps][4], bias[4];
  f32x2 last[kTaps - 1][4];      // the inputs before this one, oldest first

  __device__ __forceinline__ void load_weights(const Params &p, int c) {
    const __nv_bfloat16 *at = p.weight + static_cast<int64_t>(c / p.part) * kTaps * p.part + c % p.part;
#pragma unroll
    for (int j = 0; j < kTaps; ++j)
      pairs8(__ldg(reinterpret_cast<const uint4 *>(at + static_cast<int64_t>(j) * p.part)), w[j]);
    pairs8(p.bias ? __ldg(reinterpret_cast<const uint4 *>(p.bias + c)) : make_uint4(0, 0, 0, 0), bias);
  }
  // One token: its output, and the inputs move on.
  __device__ __forceinline__ uint4 token(const uint4 &raw, int silu) {
    f32x2 x[4];
    uint32_t y[4];
    pairs8(raw, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x2 acc = bias[i];
#pragma unroll
      for (int j = 0; j < kTaps - 1; ++j) acc = fma2(w[j][i], last[j][i], acc);
      acc = fma2(w[kTaps - 1][i], x[i], acc);
#pragma unroll
      for (int j = 0; j < kTaps - 2; ++j) last[j][i] = last[j + 1][i];
      last[kTaps - 2][i] = x[i];
      if (silu) acc = silu2(acc);
      float lo, hi;
      unpair(acc, lo, hi);
      y[i] = pack2(lo, hi);
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
  }
};

// A slot's window of 8 channels from c on: [channel][width], 8 * width elements and
// so a multiple of 16 bytes; whole vectors where the window is as wide as the taps
// before the last.
template <int kTaps, bool kF32>
__device__ __forceinline__ void read_window(const Params &p, int slot, int c,
                                            f32x2 (&last)[kTaps - 1][4]) {
  constexpr int kN = kTaps - 1, kWords = kF32 ? 8 * kN : 4 * kN;
  const int64_t at = (static_cast<int64_t>(slot) * p.channels + c) * p.width;
  if (p.width == kN) {
    uint32_t u[kWords];
    const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.window) +
                                                        at * (kF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 q = from[i];
      u[4 * i] = q.x, u[4 * i + 1] = q.y, u[4 * i + 2] = q.z, u[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = i * kN + j;
        f[i] = kF32 ? __uint_as_float(u[e])
                    : __uint_as_float(e & 1 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) last[j][i] = pair(f[2 * i], f[2 * i + 1]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t e = at + static_cast<int64_t>(i) * p.width + j;
      f[i] = kF32 ? static_cast<const float *>(p.window)[e]
                  : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.window)[e]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) last[j][i] = pair(f[2 * i], f[2 * i + 1]);
  }
}
template <int kTaps, bool kF32>
__device__ __forceinline__ void write_window(const Params &p, int slot, int c,
                                             const f32x2 (&pairs)[kTaps - 1][4]) {
  constexpr int kN = kTaps - 1, kWords = kF32 ? 8 * kN : 4 * kN;
  float last[kN][8];
#pragma unroll
  for (int j = 0; j < kN; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(pairs[j][i], last[j][2 * i], last[j][2 * i + 1]);
  const int64_t at = (static_cast<int64_t>(slot) * p.channels + c) * p.width;
  if (p.width == kN) {
    uint32_t u[kWords];
#pragma unroll
    for (int e = 0; e < kWords; ++e)
      if (kF32)
        u[e] = __float_as_uint(last[e % kN][e / kN]);
      else
        u[e] = pack2(last[2 * e % kN][2 * e / kN], last[(2 * e + 1) % kN][(2 * e + 1) / kN]);
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<char *>(p.window) + at * (kF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      to[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t e = at + static_cast<int64_t>(i) * p.width + j;
      if (kF32)
        static_cast<float *>(p.window)[e] = last[j][i];
      else
        static_cast<__nv_bfloat16 *>(p.window)[e] = __float2bfloat16_rn(last[j][i]);
    }
}

// A thread: 8 channels of a piece of a sequence.  The thread of a sequence's first
// piece reads its window and writes the new one (they may be one slot's).
template <int kTaps, bool kF32>
__global__ void __launch_bounds__(kThreads) prompt_kernel(const __grid_constant__ Params p) {
  constexpr int kN = kTaps - 1;
  follow();
  const int64_t index = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t n = index / p.vectors;
  if (n >= p.pieces) return;
  const int v = static_cast<int>(index - n * p.vectors), c = 8 * v;
  Channels<kTaps> ch;
  ch.load_weights(p, c);
  Seq seq;
  if (v == 0 && n < p.seqs.count && p.err) {         // each sequence's flags, once
    if (const int bad = resolve(p.seqs, static_cast<int>(n), &seq)) atomicOr(p.err, bad);
  }
  const int b = seq_of(p.seqs, n, kPiece);
  if (resolve(p.seqs, b, &seq)) return;
  const int64_t piece = n - (seq.start / kPiece + b), begin = piece * kPiece;
  if (piece < 0 || (piece > 0 && begin >= seq.len)) return;
  const int rows = static_cast<int>(min(static_cast<int64_t>(kPiece), seq.len - begin));
  const __nv_bfloat16 *x = p.x + seq.start * p.x_stride + c;      // the sequence's rows
  // the next rows come while these are worked on
  uint4 raw[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    if (i < rows) raw[i] = __ldg(reinterpret_cast<const uint4 *>(x + (begin + i) * p.x_stride));
  if (piece > 0) {
#pragma unroll
    for (int j = 0; j < kN; ++j)
      pairs8(__ldg(reinterpret_cast<const uint4 *>(x + (begin - kN + j) * p.x_stride)), ch.last[j]);
  } else {
    if (seq.src)
      read_window<kTaps, kF32>(p, seq.src, c, ch.last);
    else
#pragma unroll
      for (int j = 0; j < kN; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ch.last[j][i] = 0;
    if (seq.dst) {
      f32x2 next[kN][4];
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int at = seq.len - kN + j;             // of the sequence, or before it
        if (at >= 0) {
          pairs8(__ldg(reinterpret_cast<const uint4 *>(x + at * p.x_stride)), next[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            next[j][i] = ch.last[j][i];              // len 0; else `len` further
            if (j + 1 < kN && seq.len == 1) next[j][i] = ch.last[(j + 1) % kN][i];
            if (j + 2 < kN && seq.len == 2) next[j][i] = ch.last[(j + 2) % kN][i];
          }
        }
      }
      write_window<kTaps, kF32>(p, seq.dst, c, next);
    }
  }
  x += begin * p.x_stride;
  __nv_bfloat16 *out = p.output + (seq.start + begin) * p.o_stride + c;
  for (int t = 0; t < rows; t += kBatch) {
    uint4 now[kBatch];
    x += kBatch * p.x_stride;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      now[i] = raw[i];
      if (t + kBatch + i < rows) raw[i] = __ldg(reinterpret_cast<const uint4 *>(x + i * p.x_stride));
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (t + i < rows)
        *reinterpret_cast<uint4 *>(out + i * p.o_stride) = ch.token(now[i], p.silu);
    out += kBatch * p.o_stride;
  }
}

// A thread: 8 channels of a request.
template <int kTaps, bool kF32>
__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Params p) {
  follow();
  const int64_t index = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = index / p.vectors;
  if (r >= p.batch) return;
  const int v = static_cast<int>(index - r * p.vectors), c = 8 * v;
  const int slot = __ldg(p.slots + r);
  const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(p.x + r * p.x_stride + c));
  Channels<kTaps> ch;
  ch.load_weights(p, c);
  uint4 *out = reinterpret_cast<uint4 *>(p.output + r * p.o_stride + c);
  if (slot <= 0 || slot >= p.seqs.num_slots) {
    *out = make_uint4(0, 0, 0, 0);
    if (slot >= p.seqs.num_slots && p.err && v == 0) atomicOr(p.err, KDA_DEVERR_SLOT);
    return;
  }
  read_window<kTaps, kF32>(p, slot, c, ch.last);
  *out = ch.token(raw, p.silu);
  write_window<kTaps, kF32>(p, slot, c, ch.last);
}

template <class Args>
static int check(const Args *a, int64_t rows) {
  if (a->channels < 0 || a->parts < 1 || a->channels % (8 * int64_t(a->parts)) != 0)
    return KDA_ERR_SHAPE;
  if (a->taps < 2 || a->taps > 4 || rows < 0 || rows > kMostRows) return KDA_ERR_SHAPE;
  if (!stride_ok(a->x_stride, a->channels) || !stride_ok(a->o_stride, a->channels))
    return KDA_ERR_SHAPE;
  return KDA_SUCCESS;
}
template <class Args>
static Params params_of(const Args *a) {
  Params p = {};
  p.seqs.num_slots = a->num_slots;
  p.channels = a->channels;
  p.vectors = a->channels / 8;
  p.part = a->channels / a->parts;
  p.width = a->width;
  p.silu = a->silu != 0;
  p.x_stride = a->x_stride;
  p.o_stride = a->o_stride;
  p.x = static_cast<const __nv_bfloat16 *>(a->x);
  p.weight = static_cast<const __nv_bfloat16 *>(a->weight);
  p.bias = static_cast<const __nv_bfloat16 *>(a->bias);
  p.window = a->window;
  p.output = static_cast<__nv_bfloat16 *>(a->output);
  p.err = a->err;
  return p;
}
template <class Args>
static bool all_aligned(const Args *a) {
  return aligned(a->x, 16) && aligned(a->output, 16) && aligned(a->weight, 16) &&
         aligned(a->bias, 16) && aligned(a->window, 16) && aligned(a->err, 4);
}

typedef void (*Kernel)(const Params);
static Kernel prompt_of(int taps, bool f32) {
  if (taps == 2) return f32 ? prompt_kernel<2, true> : prompt_kernel<2, false>;
  if (taps == 3) return f32 ? prompt_kernel<3, true> : prompt_kernel<3, false>;
  return f32 ? prompt_kernel<4, true> : prompt_kernel<4, false>;
}
static Kernel step_of(int taps, bool f32) {
  if (taps == 2) return f32 ? step_kernel<2, true> : step_kernel<2, false>;
  if (taps == 3) return f32 ? step_kernel<3, true> : step_kernel<3, false>;
  return f32 ? step_kernel<4, true> : step_kernel<4, false>;
}

static int launch(Kernel kernel, const Params &p, int64_t threads, cudaStream_t stream) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return KDA_ERR_SHAPE;
  int dev = 0;
  DeviceFacts df;
  if (!current_device(&dev, &df)) return KDA_ERR_DEVICE;
  return launch_following(kernel, blocks, kThreads, 0, 0, stream, p) ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

static int run_prompt(const kda_conv_prompt_args *a, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  if (const int rc = check(a, a->tokens)) return rc;
  const bool pool = a->src_slots || a->dst_slots;
  if (a->seqs < 0 || a->seqs > kMostRows || (pool && a->num_slots < 1)) return KDA_ERR_SHAPE;
  if (pool && a->width < a->taps - 1) return KDA_ERR_CONV_WIDTH;
  if (a->seqs == 0 || a->channels == 0) return KDA_SUCCESS;
  if (!a->seq_starts || !a->weight || (pool && !a->window)) return KDA_ERR_NULL_POINTER;
  if (a->tokens > 0 && (!a->x || !a->output)) return KDA_ERR_NULL_POINTER;
  if (!all_aligned(a) || !aligned(a->seq_starts, 4) || !aligned(a->src_slots, 4) ||
      !aligned(a->dst_slots, 4))
    return KDA_ERR_ALIGNMENT;
  Params p = params_of(a);
  p.seqs.count = a->seqs;
  p.seqs.tokens = p.seqs.longest = a->tokens;
  p.seqs.starts = a->seq_starts;
  p.seqs.src_slots = a->src_slots;
  p.seqs.dst_slots = a->dst_slots;
  p.pieces = pieces_of(a->tokens, a->seqs, kPiece);
  return launch(prompt_of(a->taps, a->window_f32 != 0), p, p.pieces * p.vectors, stream);
}

static int run_step(const kda_conv_step_args *a, cudaStream_t stream) {
  if (!a) return KDA_ERR_NULL_ARGS;
  if (const int rc = check(a, a->batch)) return rc;
  if (a->num_slots < 1) return KDA_ERR_SHAPE;
  if (a->width < a->taps - 1) return KDA_ERR_CONV_WIDTH;
  if (a->batch == 0 || a->channels == 0) return KDA_SUCCESS;
  if (!a->x || !a->weight || !a->slots || !a->window || !a->output) return KDA_ERR_NULL_POINTER;
  if (!all_aligned(a) || !aligned(a->slots, 4)) return KDA_ERR_ALIGNMENT;
  Params p = params_of(a);
  p.slots = a->slots;
  p.batch = a->batch;
  return launch(step_of(a->taps, a->window_f32 != 0), p, static_cast<int64_t>(a->batch) * p.vectors,
                stream);
}

}  // namespace conv
}  // namespace kda

extern "C" int kda_conv_prompt(const kda_conv_prompt_args *args, void *stream) {
  return kda::conv::run_prompt(args, static_cast<cudaStream_t>(stream));
}

extern "C" int kda_conv_step(const kda_conv_step_args *args, void *stream) {
  return kda::conv::run_step(args, static_cast<cudaStream_t>(stream));
}
