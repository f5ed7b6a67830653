// Selective scan over ragged prompts.
//
// A thread holds kHeld states of a channel in registers (N / kHeld lanes a channel)
// and walks the tokens; a CTA of 128 threads takes channels of one group.  Tiles of 16
// tokens of x, dt and z come by asynchronous copies, two tiles in flight; b and c go
// through registers into FP32 in shared memory, from where every lane of a warp reads
// the same words.  What is the same for all states of a channel is computed once per
// token, two channels to an instruction, by the warp that owns the channel: the steps
// s and s x before the tile's walk, skip and gate behind it, through shared memory.
//
// Decays.  exp(s a) = ex2(s (a log2 e)) per token and state on the approximate exp2,
// and FP32 holds a factor near 1 to 2^-25: a state that remembers 1000 tokens would
// drift by 2e-5 of itself or more, to one side.  So over a tile the product of the
// factors that were used is kept too, less 1 (m <- m + q + m q, with q = e e' - 1 of two
// tokens in one operation), and at the end of two tiles the state is corrected by
// (exp(a sum s) - 1 - m) h_0, with exp - 1 from a polynomial (decay_of): 1.5 operations
// per token and state and 20 per two tiles and state, where a polynomial at every
// token would take 8.
//
// Split sequences.  A sequence much longer than an SM's share is cut into pieces:
// scan_kernel<.., false> sums each piece's own contribution to the state, from its
// end backwards (every exponent is a sum of steps, so nothing drifts there), and its
// steps; scan_kernel<.., true> runs the pieces side by side, each from the state that
// it sums up itself from the pieces before.
//
// What bounds it (GB300): the schedulers' slots.  With 16 warps an SM a token of 32
// channels x 16 states takes a warp 190 cycles of its scheduler: 75 for the products and
// sums of decays, states and outputs, 20 for the corrections' products, 12 for b and c, 6
// more for exp2 (64 of another unit, beside them), 14 for the tile's loads, 30 for the
// steps, 16 for the outputs, 7 for the corrections (each measured by leaving it out of a
// copy).  One CTA alone on an SM: 320 cycles a token with 16 states a thread, 220 with 8.
// 8 ragged sequences (9159 tokens x 4096 channels) 316 us, bound by the longest of 2047
// tokens; 32749 tokens x 4096 1079 us in 19 pieces, 390 of them in the first pass; its
// bytes would take 45 and 158.  What made it fast: 16 states a thread instead of 4 (1959
// -> 488 us, the long one 38 -> 1.5 ms), steps and outputs once per token in pairs of
// channels and without branches (488 -> 353), contributions summed backwards (1400 ->
// 1098).  Not kept: scalar operations for pairs (1174 us), exponents not ahead (1107), 2 or
// 8 tokens a walk (1124, 1127), tiles of 8 or 32 tokens (1136, 1217), 5 CTAs an SM in
// fewer registers (1240), 256 threads (1088, and 148 us instead of 117 for 1024 tokens).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <type_traits>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_ssm.cuh"

namespace kda {
namespace ssm {

constexpr int kThreads = 128;
constexpr int kTile = 16;                        // tokens

template <int kStates, int kHeld>
struct Stage {
  static constexpr int kLanes = kStates / kHeld;             // of a channel
  static constexpr int kChannels = kThreads / kLanes;        // of a CTA
  static constexpr int kOwn = 32 / kLanes;                   // of a warp
  static constexpr int kVectors = kChannels / 8;             // 16 bytes each, of a row
  static constexpr int kShared = kTile * 2 * kStates / 8;    // vectors of b and c
  __nv_bfloat16 x[2][kTile][kChannels], dt[2][kTile][kChannels], z[2][kTile][kChannels];
  float b[2][kTile][kStates], c[2][kTile][kStates];
  float2 steps[kTile][kChannels];                            // s and s x, then y
  ulonglong2 before[kHeld / 4][kThreads];                    // the states before two tiles
  // Channel c of token t of x, dt and z: odd tokens' halves of 128 bytes change places, so
  // that lanes which read two tokens' 64 bytes meet no bank twice.
  __device__ static int at(int t, int c) { return kChannels >= 64 ? c ^ ((t & 1) << 5) : c; }
};

__device__ __forceinline__ void copy16(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
}

template <int kHeld>
__device__ __forceinline__ void read_states(const float *from, f32x2 (&h)[kHeld / 2]) {
#pragma unroll
  for (int i = 0; i < kHeld / 4; ++i) {
    const float4 v = reinterpret_cast<const float4 *>(from)[i];
    h[2 * i] = pair(v.x, v.y);
    h[2 * i + 1] = pair(v.z, v.w);
  }
}
template <int kHeld>
__device__ __forceinline__ void write_states(float *to, const f32x2 (&h)[kHeld / 2]) {
#pragma unroll
  for (int i = 0; i < kHeld / 4; ++i) {
    float4 v;
    unpair(h[2 * i], v.x, v.y);
    unpair(h[2 * i + 1], v.z, v.w);
    reinterpret_cast<float4 *>(to)[i] = v;
  }
}

// A piece's start from its sequence's: over the pieces before it, h <- exp(a s) h + u with
// their steps' sums s and contributions u.
template <int kStates, int kHeld>
__device__ __forceinline__ void pass_pieces(const Params &p, int64_t first, int before, int channel,
                                            int held, const f32x2 (&a)[kHeld / 2],
                                            f32x2 (&h)[kHeld / 2]) {
  for (int j = 0; j < before; ++j) {
    const float s = p.ws_step[(first + j) * p.channels + channel];
    f32x2 u[kHeld / 2];
    read_states<kHeld>(p.ws_state + ((first + j) * p.channels + channel) * kStates + held, u);
#pragma unroll
    for (int i = 0; i < kHeld / 2; ++i) {
      float lo, hi, al, ah, ul, uh;
      unpair(h[i], lo, hi);
      unpair(a[i], al, ah);
      unpair(u[i], ul, uh);
      h[i] = pair(decayed(lo, decay_of(s * al), ul), decayed(hi, decay_of(s * ah), uh));
    }
  }
}

// h + h_0 (exp(a s) - 1 - used), for decays down to 1/2: `used` is off by 2^-24 of 1,
// which a stronger decay's own state would show, and its states remember 50 tokens.
__device__ __forceinline__ f32x2 corrected(f32x2 h, f32x2 h0, f32x2 a, float s, f32x2 product) {
  float v[2], v0[2], x[2], used[2];
  unpair(h, v[0], v[1]);
  unpair(h0, v0[0], v0[1]);
  unpair(a, x[0], x[1]);
  unpair(product, used[0], used[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float z = s * x[i];
    v[i] = fabsf(z + 0.5f) <= 0.5f ? __fmaf_rn(v0[i], less_one(z) - used[i], v[i]) : v[i];
  }
  return pair(v[0], v[1]);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// log(1 + exp(v)) of two values = max(v, 0) + log1p(e), e = exp(-|v|): as softplus(), but
// log1p(e) = e P(e), degree 8 (reweighted least squares of relative errors on [0, 1],
// 1.1e-7), as the special-function unit is busy with the decays.
__device__ __forceinline__ f32x2 softplus2(f32x2 v) {
  float lo, hi, pl, ph;
  unpair(v, lo, hi);
  const f32x2 a = pair(min_nan(fabsf(lo), 100.0f), min_nan(fabsf(hi), 100.0f));
  const f32x2 p = mul2(a, two(kLog2e)), left = fma2(a, two(-kLog2e), p);
  unpair(p, pl, ph);
  f32x2 e = pair(exp2_approx(-pl), exp2_approx(-ph));
  e = fma2(mul2(e, left), two(0.6931471806f), e);
  f32x2 t = two(5.364560522e-03f);
  t = fma2(t, e, two(-3.006473929e-02f));
  t = fma2(t, e, two(7.920283079e-02f));
  t = fma2(t, e, two(-1.375365853e-01f));
  t = fma2(t, e, two(1.915358752e-01f));
  t = fma2(t, e, two(-2.485714704e-01f));
  t = fma2(t, e, two(3.332132101e-01f));
  t = fma2(t, e, two(-4.999964833e-01f));
  t = fma2(t, e, two(1.000000000e+00f));
  return fma2(e, t, pair(max_nan(lo, 0.0f), max_nan(hi, 0.0f)));
}

template <int kStates, int kHeld, bool kOut>
__global__ void __launch_bounds__(kThreads, kHeld == 16 ? 4 : 6) scan_kernel(const __grid_constant__ Params p) {
  using S = Stage<kStates, kHeld>;
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

  // x, dt and z of a tile: this thread's vectors are kStep tokens apart
  constexpr int kStep = kThreads / S::kVectors < kTile ? kThreads / S::kVectors : kTile;
  constexpr int kCopies = kTile / kStep;
  static_assert(kThreads % S::kVectors == 0 && kTile % kStep == 0, "whole rows");
  const int copy_t = tid / S::kVectors, copy_c = tid % S::kVectors * 8;
  const int copy_to = copy_c < wide && copy_t < kStep ? rows - copy_t : 0;        // the first token that is not there
  const __nv_bfloat16 *from_x = p.x + (row0 + copy_t) * p.x_stride + channel0 + copy_c;
  const __nv_bfloat16 *from_dt = p.dt + (row0 + copy_t) * p.dt_stride + channel0 + copy_c;
  const __nv_bfloat16 *from_z =
      kOut && p.z ? p.z + (row0 + copy_t) * p.z_stride + channel0 + copy_c : nullptr;
  auto load = [&](int tile) {
    const int buf = tile & 1;
    const int64_t rows_before = static_cast<int64_t>(tile) * kTile;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const int t = copy_t + k * kStep, c = S::at(t, copy_c);
      if (tile * kTile + k * kStep < copy_to) {
        copy16(&st.x[buf][t][c], from_x + (rows_before + k * kStep) * p.x_stride);
        copy16(&st.dt[buf][t][c], from_dt + (rows_before + k * kStep) * p.dt_stride);
        if (kOut && from_z) copy16(&st.z[buf][t][c], from_z + (rows_before + k * kStep) * p.z_stride);
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

  const int tiles = (rows + kTile - 1) / kTile;
  if (rows > 0) {                                  // contributions are summed from the end
    load(kOut ? 0 : tiles - 1);
    fetch(kOut ? 0 : tiles - 1);
  }
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
  // for what is once a token: two channels, every kStride-th token, of this lane
  constexpr int kPairs = S::kOwn / 2, kStride = 32 / kPairs;
  const int lane = tid & 31, own = (tid >> 5) * S::kOwn, at2 = own + lane % kPairs * 2;
  const int t2 = lane / kPairs;
  const bool live2 = at2 < wide;
  f32x2 skip = 0, bias = 0;
  if (live2) {
    const int c = channel0 + at2;
    if (p.d) skip = pair(__ldg(p.d + c), __ldg(p.d + c + 1));
    if (p.dt_bias) bias = pair(__ldg(p.dt_bias + c), __ldg(p.dt_bias + c + 1));
  }
#pragma unroll
  for (int i = 0; i < kHeld / 2; ++i) h[i] = 0;
  // A split sequence's last piece leaves no contribution: its place holds the first
  // state for the pass with outputs, whose last piece may write over it in the pool.
  const int last = p.piece > 0 && seq.len > 0 ? (seq.len - 1) / p.piece : 0;
  float *const copy = p.ws_state + ((first + last) * p.channels + channel) * kStates + held;
  if (kOut && last > 0) {
    if (seq.src) read_states<kHeld>(copy, h);
    pass_pieces<kStates, kHeld>(p, first, piece, channel, held, a, h);
  } else if (seq.src && piece == 0) {
    read_states<kHeld>(state_of(p, seq.src, channel, kStates) + held, h);
    if (!kOut) {
      if (live) write_states<kHeld>(copy, h);
#pragma unroll
      for (int i = 0; i < kHeld / 2; ++i) h[i] = 0;
    }
  }
  float sum = 0.0f;                                // steps of two tiles, or of the piece
  f32x2 used[kHeld / 2];
  __nv_bfloat16 *out = kOut ? p.output + (row0 + t2) * p.o_stride + channel0 + at2 : nullptr;

  for (int i = 0; i < tiles; ++i) {
    const int tile = kOut ? i : tiles - 1 - i;
    const int buf = tile & 1, count = min(kTile, rows - tile * kTile);
    copies_done();
    spread(tile);
    __syncthreads();
    if (i + 1 < tiles) {
      load(kOut ? tile + 1 : tile - 1);
      fetch(kOut ? tile + 1 : tile - 1);
    }
    if (kOut && (tile & 1) == 0) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kHeld / 2; i += 2) {
        st.before[i / 2][tid] = make_ulonglong2(h[i], h[i + 1]);
        used[i] = used[i + 1] = 0;
      }
    }
    // (rows behind the piece's end and channels behind the group's: what is there is
    // computed with, and goes nowhere)
    auto steps_of = [&](auto soft) {
#pragma unroll
      for (int k = 0; k < kTile / kStride; ++k) {
        const int t = t2 + k * kStride;
        const f32x2 x = unpack2(*reinterpret_cast<const uint32_t *>(&st.x[buf][t][S::at(t, at2)]));
        f32x2 v = add2(unpack2(*reinterpret_cast<const uint32_t *>(&st.dt[buf][t][S::at(t, at2)])), bias);
        if (decltype(soft)::value) v = softplus2(v);
        float4 w;
        unpair(v, w.x, w.z);
        unpair(mul2(v, x), w.y, w.w);
        *reinterpret_cast<float4 *>(&st.steps[t][at2]) = w;
      }
    };
    if (p.softplus)
      steps_of(std::true_type());
    else
      steps_of(std::false_type());
    __syncwarp();
    // kMany tokens at a time: what they add up to leaves the registers behind them,
    // so that the next one's loads and exponents need not wait for a store
    auto walk = [&](int t0, auto many) {
      constexpr int kMany = decltype(many)::value;
      float2 w[kMany];
      float ys[kMany];
#pragma unroll
      for (int u = 0; u < kMany; ++u) w[u] = st.steps[t0 + u][mine];
      auto decay = [&](float s, int i) {
        float lo, hi;
        unpair(mul2(two(s), a[i]), lo, hi);
        return pair(exp2_approx(lo), exp2_approx(hi));
      };
      f32x2 e[kHeld / 2], last[kHeld / 2];
#pragma unroll
      for (int i = 0; i < kHeld / 2; ++i) e[i] = decay(w[0].x, i);
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        const int t = t0 + u;
        sum += w[u].x;
        const f32x2 sx = two(w[u].y);
        const ulonglong2 *bn = reinterpret_cast<const ulonglong2 *>(st.b[buf][t] + held);
        const ulonglong2 *cn = reinterpret_cast<const ulonglong2 *>(st.c[buf][t] + held);
        f32x2 y[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kHeld / 2; i += 2) {
          const ulonglong2 bb = bn[i / 2], cc = cn[i / 2];
#pragma unroll
          for (int k = i; k < i + 2; ++k) {
            const f32x2 now = e[k];
            if (u + 1 < kMany) e[k] = decay(w[u + 1].x, k);      // the next token's, ahead
            if (u & 1) {                             // two tokens: m (q + 1) + q, q = e e - 1
              const f32x2 q = fma2(last[k], now, two(-1.0f));
              used[k] = add2(fma2(used[k], q, q), used[k]);
            } else if (u + 1 == kMany) {
              used[k] = fma2(used[k], now, add2(now, two(-1.0f)));
            } else {
              last[k] = now;
            }
            h[k] = fma2(h[k], now, mul2(sx, k == i ? bb.x : bb.y));
            y[k - i] = fma2(h[k], k == i ? cc.x : cc.y, y[k - i]);
          }
        }
        float lo, hi;
        unpair(add2(y[0], y[1]), lo, hi);
        ys[u] = lo + hi;
      }
#pragma unroll
      for (int o = 1; o < S::kLanes; o <<= 1)
#pragma unroll
        for (int u = 0; u < kMany; ++u) ys[u] += __shfl_xor_sync(0xffffffffu, ys[u], o);
      if (S::kLanes > 1) __syncwarp();                 // all lanes of the channel have read w
#pragma unroll
      for (int u = 0; u < kMany; ++u)
        if (held == 0) st.steps[t0 + u][mine].x = ys[u];
    };
    // A piece's contribution: sum_t exp(a sum of the steps behind t) s_t x_t b_t.
    auto gather = [&](int t0, auto many) {
      constexpr int kMany = decltype(many)::value;
      float2 w[kMany];
#pragma unroll
      for (int u = 0; u < kMany; ++u) w[u] = st.steps[t0 - u][mine];
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        const ulonglong2 *bn = reinterpret_cast<const ulonglong2 *>(st.b[buf][t0 - u] + held);
#pragma unroll
        for (int i = 0; i < kHeld / 2; i += 2) {
          const ulonglong2 bb = bn[i / 2];
#pragma unroll
          for (int k = i; k < i + 2; ++k) {
            float lo, hi;
            unpair(mul2(two(sum), a[k]), lo, hi);
            h[k] = fma2(pair(exp2_approx(lo), exp2_approx(hi)), mul2(two(w[u].y), k == i ? bb.x : bb.y),
                        h[k]);
          }
        }
        sum += w[u].x;
      }
    };
    if (kOut) {
      int t = 0;
#pragma unroll 1
      for (; t + 4 <= count; t += 4) walk(t, std::integral_constant<int, 4>());
#pragma unroll 1
      for (; t < count; ++t) walk(t, std::integral_constant<int, 1>());
    } else {
      int t = count - 1;
#pragma unroll 1
      for (; t >= 3; t -= 4) gather(t, std::integral_constant<int, 4>());
#pragma unroll 1
      for (; t >= 0; --t) gather(t, std::integral_constant<int, 1>());
      __syncwarp();
    }
    if (kOut) {
      __syncwarp();
      const int ends = live2 ? count : 0;
      const int64_t step = kStride * p.o_stride;
      auto outputs = [&](auto gated) {
#pragma unroll
        for (int k = 0; k < kTile / kStride; ++k) {
          const int t = t2 + k * kStride;
          const float4 w = *reinterpret_cast<const float4 *>(&st.steps[t][at2]);
          const f32x2 x = unpack2(*reinterpret_cast<const uint32_t *>(&st.x[buf][t][S::at(t, at2)]));
          f32x2 y = fma2(skip, x, pair(w.x, w.z));
          if (decltype(gated)::value)
            y = mul2(y, silu2(unpack2(*reinterpret_cast<const uint32_t *>(&st.z[buf][t][S::at(t, at2)]))));
          float lo, hi;
          unpair(y, lo, hi);
          if (t < ends) *reinterpret_cast<uint32_t *>(out + k * step) = pack2(lo, hi);
        }
      };
      if (p.z)
        outputs(std::true_type());
      else
        outputs(std::false_type());
      out += kTile * p.o_stride;
      __syncwarp();
    }
    if (kOut && ((tile & 1) || i + 1 == tiles)) {
#pragma unroll
      for (int i = 0; i < kHeld / 2; i += 2) {
        const ulonglong2 h0 = st.before[i / 2][tid];
        h[i] = corrected(h[i], h0.x, a[i], sum, used[i]);
        h[i + 1] = corrected(h[i + 1], h0.y, a[i + 1], sum, used[i + 1]);
      }
    }
  }
  if (!live) return;
  float *to = nullptr;
  if (!kOut) {
    to = p.ws_state + (n * p.channels + channel) * kStates + held;
    if (held == 0) p.ws_step[n * p.channels + channel] = sum;
  } else if (seq.dst && row0 + rows == seq.start + seq.len) {
    to = state_of(p, seq.dst, channel, kStates) + held;
  }
  if (to) write_states<kHeld>(to, h);
}

template <int kStates, int kHeld>
// (Not launched to start ahead of the end of the kernel before, as the others: CTAs then go
// where that one leaves room first, several long sequences to an SM: ragged 316 -> 438 us.)
static int launch(Params &p, cudaStream_t stream, int dev) {
  using S = Stage<kStates, kHeld>;
  p.group_blocks = (p.span + S::kChannels - 1) / S::kChannels;
  p.blocks = p.channels / p.span * p.group_blocks;
  const int64_t units = p.piece > 0 ? pieces_of(p.seqs.tokens, p.seqs.count, p.piece) : p.seqs.count;
  if (units * p.blocks > 0x7fffffffll) return KDA_ERR_SHAPE;
  static std::atomic<bool> out_done[kMaxDevices];
  if (!set_smem_limit_once(out_done, dev, reinterpret_cast<const void *>(scan_kernel<kStates, kHeld, true>),
                           sizeof(S)))
    return KDA_ERR_LAUNCH;
  const int grid = static_cast<int>(units * p.blocks);
  if constexpr (kHeld == 16) {
    if (p.piece > 0) {
      static std::atomic<bool> sum_done[kMaxDevices];
      if (!set_smem_limit_once(sum_done, dev,
                               reinterpret_cast<const void *>(scan_kernel<kStates, kHeld, false>), sizeof(S)))
        return KDA_ERR_LAUNCH;
      scan_kernel<kStates, kHeld, false><<<grid, kThreads, sizeof(S), stream>>>(p);
      if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH;
    }
  }
  scan_kernel<kStates, kHeld, true><<<grid, kThreads, sizeof(S), stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

template <int kHeld>
static int launch_of(Params &p, int states, int dev, cudaStream_t stream) {
  return states == 16 ? launch<16, kHeld>(p, stream, dev)
                      : states == 32 ? launch<32, kHeld>(p, stream, dev)
                                     : launch<64, kHeld>(p, stream, dev);
}

int launch_prompt(Params &p, int states, int held, int dev, cudaStream_t stream) {
  return held == 8 ? launch_of<8>(p, states, dev, stream) : launch_of<16>(p, states, dev, stream);
}

}  // namespace ssm
}  // namespace kda
