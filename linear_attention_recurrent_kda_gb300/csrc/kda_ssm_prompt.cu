// Selective scan over ragged prompts.
//
// A CTA of 256 threads takes channels of one group.  128 of them walk the tokens, each
// with kHeld states of a channel in registers (N / kHeld lanes a channel) and no more
// than that; 128 helpers do for tiles of 16 tokens, one ahead and one behind the walk,
// what is the same for all states of a channel: x, dt and z by asynchronous copies, two
// tiles in flight, b and c through registers into FP32 in shared memory, from where every
// lane of a warp reads the same words, the steps s and s x, skip and gate, two channels to
// an instruction.  The walk waits for them 26 cycles a tile.
//
// Decays.  exp(s a) = ex2(s (a log2 e)) per token and state on the approximate exp2,
// and FP32 holds a factor near 1 to 2^-25: a state that remembers 1000 tokens would
// drift by 2e-5 of itself or more, to one side.  So over a tile the product of the
// factors that were used is kept too, less 1 (m <- m + q + m q, with q = e e' - 1 of two
// tokens in one operation), and at the end of two tiles the state is corrected by
// (exp(a sum s) - 1 - m) h_0, with exp - 1 from a polynomial (less_one): 1.5 operations
// per token and state and 20 per two tiles and state, where a polynomial at every
// token would take 8.
//
// Split sequences.  A sequence much longer than an SM's share is cut into pieces:
// scan_kernel<.., false> sums each piece's own contribution to the state, from its
// end backwards (every exponent is a sum of steps, so nothing drifts there), and its
// steps; scan_kernel<.., true> runs the pieces side by side, each from the state that
// it sums up itself from the pieces before.
//
// What bounds it (GB300): where SMs are full, the schedulers' slots and the FP32 pipe: a
// token of 32 channels x 16 states takes 190 cycles of a scheduler, 134 of them
// instructions: 75 for the products and sums of decays, states and outputs and exp2, 20 for
// the corrections' products, 12 for b and c, and what the helpers do.  Where CTAs are few, a
// CTA's own time: 135 cycles a token with 8 states a thread, 230 with 16.
// 8 ragged sequences (9159 tokens x 4096 channels) 237 us, one of 1024 x 4096 62 us (74
// whole), 32749 tokens x 4096 1081 us in 28 pieces, 400 of them in the first pass; the
// ragged ones' bytes would take 45, the long one's 158.  What made it fast: 16 states a
// thread instead of 4 (1959 -> 488 us, the long one 38 -> 1.5 ms), steps and outputs once per
// token in pairs of channels and without branches (488 -> 353), contributions summed
// backwards (1400 -> 1098), helpers (316 -> 250, 1024 tokens whole 115 -> 76; before, each
// warp did its own channels' steps and outputs between the walks of its tiles), a whole
// tile's walk unrolled with 8 states (250 -> 242), its lanes' sums added by the helpers (242
// -> 236).  Not kept: scalar operations for pairs
// (1174 us; for some of them 1081 to 1110), exponents not ahead (1107), 2 or 8 tokens a walk
// with 16 states (1124, 1127), tiles of 8 or 32 tokens (1136, 1217).
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
// Sequences up to here: the kernel may start while the one before it ends.  CTAs then go
// where that one leaves room first, and long sequences meet on an SM (the ragged ones above
// 316 -> 438 us, before the helpers were).
constexpr int kAhead = 64;

template <int kStates, int kHeld>
struct Stage {
  static constexpr int kLanes = kStates / kHeld;             // of a channel
  static constexpr int kChannels = kThreads / kLanes;        // of a CTA
  static constexpr int kVectors = kChannels / 8;             // 16 bytes each, of a row
  static constexpr int kShared = kTile * 2 * kStates / 8;    // vectors of b and c
  __nv_bfloat16 x[3][kTile][kChannels], dt[2][kTile][kChannels], z[2][kTile][kChannels];
  float b[2][kTile][kStates], c[2][kTile][kStates];
  float2 steps[2][kTile][kChannels];                         // s and s x, then y
  ulonglong2 before[kHeld / 4][kThreads];                    // the states before two tiles
};

// Named barriers of all threads: a tile's steps, b and c are there (the helpers arrive),
// its outputs are (the walkers do); two of each in turn.  And one of the helpers.
constexpr int kReady = 1, kDone = 3, kHelpers = 5;
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(2 * kThreads) : "memory");
}
__device__ __forceinline__ void bar_helpers() {
  asm volatile("bar.sync %0, %1;" ::"n"(kHelpers), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void bar_wait(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(2 * kThreads) : "memory");
}

__device__ __forceinline__ void copy16(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
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
      h[i] = pair(decayed(lo, s * al, ul), decayed(hi, s * ah, uh));
    }
  }
}

// h + h_0 (exp(a s) - 1 - used), for decays down to 1/2: `used` is off by 2^-24 of 1,
// which a stronger decay's own state would show, and its states remember 50 tokens.  (An
// infinite h_0 has nothing to correct.)
__device__ __forceinline__ f32x2 corrected(f32x2 h, f32x2 h0, f32x2 a, float s, f32x2 product) {
  float v[2], v0[2], x[2], used[2];
  unpair(h, v[0], v[1]);
  unpair(h0, v0[0], v0[1]);
  unpair(a, x[0], x[1]);
  unpair(product, used[0], used[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float z = s * x[i];
    v[i] = fabsf(z + 0.5f) <= 0.5f && fabsf(v0[i]) < INFINITY ? __fmaf_rn(v0[i], less_one(z) - used[i], v[i]) : v[i];
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
__global__ void __launch_bounds__(2 * kThreads, 3) scan_kernel(const __grid_constant__ Params p) {
  using S = Stage<kStates, kHeld>;
  extern __shared__ __align__(16) uint8_t raw[];
  S &st = *reinterpret_cast<S *>(raw);
  follow();
  const int block = blockIdx.x % p.blocks;
  const int64_t n = blockIdx.x / p.blocks;
  const int group = block / p.group_blocks;
  const int channel0 = group * p.span + (block - group * p.group_blocks) * S::kChannels;
  const int wide = min(S::kChannels, (group + 1) * p.span - channel0);   // channels, 8 at least
  const int tid = threadIdx.x % kThreads, mine = tid / S::kLanes, held = tid % S::kLanes * kHeld;
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
  const int tiles = (rows + kTile - 1) / kTile;
  // (launched with 80 registers a thread, 3 CTAs an SM: 104 + 56 for a walker and a helper)
  if (threadIdx.x >= kThreads) {                   // a helper
    regs_dec<56>();
    // x, dt and z of a tile: this thread's vectors are kStep tokens apart
    constexpr int kStep = kThreads / S::kVectors < kTile ? kThreads / S::kVectors : kTile;
    constexpr int kCopies = kTile / kStep;
    static_assert(kThreads % S::kVectors == 0 && kTile % kStep == 0, "whole rows");
    const int copy_t = tid / S::kVectors, copy_c = tid % S::kVectors * 8;
    const int copy_to = copy_c < wide && copy_t < kStep ? rows - copy_t : 0;   // tokens from there on are not
    const __nv_bfloat16 *from_x = p.x + (row0 + copy_t) * p.x_stride + channel0 + copy_c;
    const __nv_bfloat16 *from_dt = p.dt + (row0 + copy_t) * p.dt_stride + channel0 + copy_c;
    const __nv_bfloat16 *from_z =
        kOut && p.z ? p.z + (row0 + copy_t) * p.z_stride + channel0 + copy_c : nullptr;
    auto load = [&](int tile, int stage, int buf) {
      const int64_t rows_before = static_cast<int64_t>(tile) * kTile;
#pragma unroll
      for (int k = 0; k < kCopies; ++k) {
        const int t = copy_t + k * kStep;
        if (tile * kTile + k * kStep < copy_to) {
          copy16(&st.x[stage][t][copy_c], from_x + (rows_before + k * kStep) * p.x_stride);
          copy16(&st.dt[buf][t][copy_c], from_dt + (rows_before + k * kStep) * p.dt_stride);
        }
      }
    };
    auto load_gate = [&](int tile) {
      if (!kOut || !from_z) return;
      const int64_t rows_before = static_cast<int64_t>(tile) * kTile;
#pragma unroll
      for (int k = 0; k < kCopies; ++k)
        if (tile * kTile + k * kStep < copy_to)
          copy16(&st.z[tile & 1][copy_t + k * kStep][copy_c], from_z + (rows_before + k * kStep) * p.z_stride);
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
    auto spread = [&](int buf) {
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int i = tid + k * kThreads, t = i / (kStates / 4), v = i % (kStates / 4);
        if (i < S::kShared) {
          float f[8];
          unpack8(shared[k], f);
          float4 *to = reinterpret_cast<float4 *>(
              (v < kStates / 8 ? st.b[buf][t] : st.c[buf][t]) + v % (kStates / 8) * 8);
          to[0] = make_float4(f[0], f[1], f[2], f[3]);
          to[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
    };

    // two channels of every kStride-th token
    constexpr int kPairs = S::kChannels / 2, kStride = kThreads / kPairs;
    const int at2 = tid % kPairs * 2, t2 = tid / kPairs;
    const bool live2 = at2 < wide;
    f32x2 skip = 0, bias = 0;
    if (live2) {
      const int c = channel0 + at2;
      if (p.d) skip = pair(__ldg(p.d + c), __ldg(p.d + c + 1));
      if (p.dt_bias) bias = pair(__ldg(p.dt_bias + c), __ldg(p.dt_bias + c + 1));
    }
    // (rows behind the piece's end and channels behind the group's: what is there is
    // computed with, and goes nowhere)
    auto steps = [&](int buf, int stage) {
      auto steps_of = [&](auto soft) {
#pragma unroll
        for (int k = 0; k < kTile / kStride; ++k) {
          const int t = t2 + k * kStride;
          const f32x2 x = unpack2(*reinterpret_cast<const uint32_t *>(&st.x[stage][t][at2]));
          f32x2 v = add2(unpack2(*reinterpret_cast<const uint32_t *>(&st.dt[buf][t][at2])), bias);
          if (decltype(soft)::value) v = softplus2(v);
          float4 w;
          unpair(v, w.x, w.z);
          unpair(mul2(v, x), w.y, w.w);
          *reinterpret_cast<float4 *>(&st.steps[buf][t][at2]) = w;
        }
      };
      if (p.softplus)
        steps_of(std::true_type());
      else
        steps_of(std::false_type());
    };
    auto results = [&](int tile, int buf, int stage) {
      const int count = min(kTile, rows - tile * kTile);
      __nv_bfloat16 *const to =
          p.output + (row0 + static_cast<int64_t>(tile) * kTile + t2) * p.o_stride + channel0 + at2;
      const int ends = live2 ? count : 0;
      const int64_t step = kStride * p.o_stride;
      auto outputs = [&](auto gated) {
#pragma unroll
        for (int k = 0; k < kTile / kStride; ++k) {
          const int t = t2 + k * kStride;
          const float4 w = *reinterpret_cast<const float4 *>(&st.steps[buf][t][at2]);
          const f32x2 x = unpack2(*reinterpret_cast<const uint32_t *>(&st.x[stage][t][at2]));
          f32x2 y = fma2(skip, x, S::kLanes == 1 ? pair(w.x, w.z) : pair(w.x + w.y, w.z + w.w));
          if (decltype(gated)::value)
            y = mul2(y, silu2(unpack2(*reinterpret_cast<const uint32_t *>(&st.z[buf][t][at2]))));
          float lo, hi;
          unpair(y, lo, hi);
          if (t < ends) *reinterpret_cast<uint32_t *>(to + k * step) = pack2(lo, hi);
        }
      };
      if (p.z)
        outputs(std::true_type());
      else
        outputs(std::false_type());
    };
    auto tile_of = [&](int i) { return kOut ? i : tiles - 1 - i; };   // contributions: from the end
    if (tiles > 0) {
      load(tile_of(0), 0, 0);
      fetch(tile_of(0));
      copies_done();
      bar_helpers();
      load_gate(0);
      if (tiles > 1) load(tile_of(1), 1, 1);
    }
    for (int i = 0, stage = 0; i < tiles; ++i) {   // stage: i % 3
      const int next = stage == 2 ? 0 : stage + 1, before = stage == 0 ? 2 : stage - 1;
      spread(i & 1);
      if (i + 1 < tiles) fetch(tile_of(i + 1));
      steps(i & 1, stage);
      bar_arrive(kReady + (i & 1));
      if (i > 0) {
        bar_wait(kDone + ((i - 1) & 1));
        if (kOut) results(i - 1, (i - 1) & 1, before);
      }
      if (i + 1 < tiles) {
        copies_done();
        bar_helpers();                             // of tile i + 1, by all; tile i - 1 is read
        load_gate(i + 1);
        if (i + 2 < tiles) load(tile_of(i + 2), before, i & 1);
      } else {
        if (kOut) {
          copies_done();                           // the last gate
          bar_helpers();
        }
        bar_wait(kDone + (i & 1));
        if (kOut) results(i, i & 1, stage);
      }
      stage = next;
    }
    return;
  }
  regs_inc<104>();
  const bool live = mine < wide;
  const int channel = channel0 + (live ? mine : 0);

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

  for (int i = 0; i < tiles; ++i) {
    const int tile = kOut ? i : tiles - 1 - i;
    const int buf = i & 1, count = min(kTile, rows - tile * kTile);
    bar_wait(kReady + buf);
    if (kOut && (tile & 1) == 0) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kHeld / 2; i += 2) {
        st.before[i / 2][tid] = make_ulonglong2(h[i], h[i + 1]);
        used[i] = used[i + 1] = 0;
      }
    }
    // kMany tokens at a time: what they add up to leaves the registers behind them,
    // so that the next one's loads and exponents need not wait for a store
    auto walk = [&](int t0, auto many) {
      constexpr int kMany = decltype(many)::value;
      float2 w[kMany];
      float ys[kMany];
#pragma unroll
      for (int u = 0; u < kMany; ++u) w[u] = st.steps[buf][t0 + u][mine];
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
        f32x2 y = 0;
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
            y = k == 0 ? mul2(h[k], cc.x) : fma2(h[k], k == i ? cc.x : cc.y, y);
          }
        }
        float lo, hi;
        unpair(y, lo, hi);
        ys[u] = lo + hi;
      }
#pragma unroll
      for (int o = 2; o < S::kLanes; o <<= 1)
#pragma unroll
        for (int u = 0; u < kMany; ++u) ys[u] += __shfl_xor_sync(0xffffffffu, ys[u], o);
      if (S::kLanes > 1) __syncwarp();                 // all lanes of the channel have read w
#pragma unroll
      for (int u = 0; u < kMany; ++u)
        if (S::kLanes == 1)
          st.steps[buf][t0 + u][mine].x = ys[u];
        else if (held < 2 * kHeld)                     // two lanes' sums, which a helper adds
          (&st.steps[buf][t0 + u][mine].x)[held / kHeld] = ys[u];
    };
    // A piece's contribution: sum_t exp(a sum of the steps behind t) s_t x_t b_t.
    auto gather = [&](int t0, auto many) {
      constexpr int kMany = decltype(many)::value;
      float2 w[kMany];
#pragma unroll
      for (int u = 0; u < kMany; ++u) w[u] = st.steps[buf][t0 - u][mine];
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
      if (kHeld == 8 && count == kTile) {
        walk(0, std::integral_constant<int, kTile>());
        t = kTile;
      }
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
    }
    bar_arrive(kDone + buf);
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
static int launch(Params &p, cudaStream_t stream, int dev) {
  using S = Stage<kStates, kHeld>;
  p.group_blocks = (p.span + S::kChannels - 1) / S::kChannels;
  p.blocks = p.channels / p.span * p.group_blocks;
  const int64_t units = p.piece > 0 ? pieces_of(p.seqs.tokens, p.seqs.count, p.piece) : p.seqs.count;
  static std::atomic<bool> out_done[kMaxDevices];
  if (!set_smem_limit_once(out_done, dev, reinterpret_cast<const void *>(scan_kernel<kStates, kHeld, true>),
                           sizeof(S)))
    return KDA_ERR_LAUNCH;
  const int grid = static_cast<int>(units * p.blocks);     // (that it is one: plan_prompt)
  if constexpr (kHeld == 16) {
    if (p.piece > 0) {
      static std::atomic<bool> sum_done[kMaxDevices];
      if (!set_smem_limit_once(sum_done, dev,
                               reinterpret_cast<const void *>(scan_kernel<kStates, kHeld, false>), sizeof(S)))
        return KDA_ERR_LAUNCH;
      scan_kernel<kStates, kHeld, false><<<grid, 2 * kThreads, sizeof(S), stream>>>(p);
      if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH;
    }
  }
  if (p.seqs.longest <= kAhead)
    return launch_following(scan_kernel<kStates, kHeld, true>, grid, 2 * kThreads, sizeof(S), 0, stream, p)
               ? KDA_SUCCESS
               : KDA_ERR_LAUNCH;
  scan_kernel<kStates, kHeld, true><<<grid, 2 * kThreads, sizeof(S), stream>>>(p);
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
