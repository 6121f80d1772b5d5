// gdn_conv_step.cu -- the causal convolution + SiLU on a pool of windows, for generation: the
// next tokens of N sequences, the last W-1 rows of each kept in its slot.
//   z[t, c] = b[c] + sum_i w[c, i] row(t - (W-1) + i)[c],  y = z sigma(z)
// with row(s) the token s of the sequence, or its window's row before the first token.
//
// Bandwidth-bound.  Three ways:
//   - one token each (no cu_seqlens): a thread owns two channels and takes the sequences gridDim.y apart, its
//     taps in registers.  All that does not hang on the slot is requested at once, so that a call is two
//     loads deep;
//   - short sequences among any: a thread owns four channels of one sequence, and asks for four tokens at a time;
//   - any lengths: a thread owns four channels and walks a range of tokens with the last W-1 rows in registers,
//     the next rows on their way into shared memory (each thread copies what it reads, so no thread waits
//     for another).
//
// Long sequences are cut over CTAs, and a slot may be read and written by the same call, so whatever
// reads or writes a sequence's slots is done by one CTA per channel block, the one whose range holds its first
// token (a short one's own CTA): it also computes the first W-1 tokens, which need the window (past its range's end if they lie
// there), and writes the windows of all the sequence's tokens from its own copy of the old window and x.
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_prof.h"

namespace gdn {

constexpr int CS_THREADS = 128;
constexpr int CS_THREADS1 = 128;  // of a CTA of the kernel for single tokens
constexpr int CS_VEC = 4;         // channels per thread, and of the kernel for single tokens:
constexpr int CS_VEC1 = 2;
constexpr int CS_STAGES = 16;     // rows of a thread on their way
constexpr int CS_FEW = 4;         // tokens of a short sequence that a thread has in registers
constexpr int CS_SHORT = 16;      // tokens up to which a sequence of many is a thread's own
constexpr int CS_MEAN = 8;        // where the mean is no more than so many
constexpr int CS_LOOK = 4;        // slot numbers a lane has requested together
// CTAs an SM that make a round: of the range kernel for 16-bit rows what it holds.  It holds 6 for FP32 rows (32 KiB of ring
// each) and 6 or 4 of the mixed kernel, but with 6 ranges are as quick or slower there, too (9 FP32 sequences of up to
// 693 tokens of 1,128 channels 9.4 us, with 7 8.9; 29 of up to 106 of 8,608 20.3 and 19.5; 64 of 1-4 of 10,240 6.8 both).
constexpr int CS_ROUND = 7;
constexpr int CS_ROUND1 = 12;     // that an SM holds of the kernel for single tokens
constexpr int CS_LONG = 64;       // tokens of a long range
constexpr int CS_MAXR = 256;      // tokens per range, at most, while the grid has rows for so many ranges:
constexpr int CS_ROWS = 65535;

struct ConvStepArgs {
  const void* x;
  const float* w;
  const float* b;
  const int* cu;
  const int* slot_in;
  const int* slot_out;
  void* window;
  void* y;
  int* err;
  int64_t xs, ys;
  int T, N, C, slots;
  int R;   // tokens of a range; with single tokens the sequences that a thread has at a time
};

// z sigma(z), with the hardware's exponential and reciprocal: within (1.25 |z| + 8) 2^-24 of the value (the exponential's
// argument is rounded once), down to -87, and zero where y is less than 2^-119. That is far below 16-bit rows' rounding; for
// FP32 rows it is a choice: the far negative values, which lose the most places, are nothing next to a row's others (y of random
// rows is 6.7e-8 of its norm from FP64, that of elementary FP32 operations 7.4e-8), and CUDA's expf and division take
// 475 us for 360 (28,924 ragged tokens of 10,240 channels).
__device__ __forceinline__ float silu(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504088896f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return z * r;
}

// The last sequence n with cu[n] <= t (0 if there is none), found by a whole warp: 32 probes a step.
__device__ __forceinline__ int sequence_of(const int* cu, int N, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = N;   // the answer lies in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lo + lane * step;
    const bool in = lane * step < len && cu[at] <= t;
    const unsigned m = __ballot_sync(~0u, in);
    const int top = m ? 31 - __clz(m) : 0;
    len = min(step, len - top * step);
    lo += top * step;
  }
  return lo;
}

// taps and bias of V channels from c0 on, as pairs of channels
template <int W, int V> struct Taps {
  float2 w[W][V / 2], b[V / 2];
  __device__ __forceinline__ void load(const ConvStepArgs& a, int c0) {
    const float* wp = a.w + (int64_t)c0 * W;   // (c0 is a multiple of V)
    float t[V * W];
    if constexpr (V * W % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V * W / 4; ++i) {
        const float4 f = reinterpret_cast<const float4*>(wp)[i];
        t[4 * i] = f.x;
        t[4 * i + 1] = f.y;
        t[4 * i + 2] = f.z;
        t[4 * i + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V * W / 2; ++i) {
        const float2 f = reinterpret_cast<const float2*>(wp)[i];
        t[2 * i] = f.x;
        t[2 * i + 1] = f.y;
      }
    }
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i][e] = make_float2(t[2 * e * W + i], t[(2 * e + 1) * W + i]);
      b[e] = a.b ? reinterpret_cast<const float2*>(a.b + c0)[e] : make_float2(0.f, 0.f);
    }
  }
};
template <typename E, int V> __device__ __forceinline__ void as_pairs(const RawV<E, V>& r, float2 (&h)[V / 2]) {
  float f[V];
  r.get(f);
#pragma unroll
  for (int e = 0; e < V / 2; ++e) h[e] = make_float2(f[2 * e], f[2 * e + 1]);
}
// y of one row after hist (the W-1 rows before, the newest last), of which it becomes the newest
template <typename E, int W, int V>
__device__ __forceinline__ RawV<E, V> conv_row(const Taps<W, V>& k, const RawV<E, V>& row,
                                               float2 (&hist)[W > 1 ? W - 1 : 1][V / 2]) {
  float z[V];
  float2 now[V / 2];
  as_pairs(row, now);
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    float2 s = k.b[e];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) s = __ffma2_rn(k.w[i][e], hist[i][e], s);
    s = __ffma2_rn(k.w[W - 1][e], now[e], s);
    z[2 * e] = silu(s.x);
    z[2 * e + 1] = silu(s.y);
#pragma unroll
    for (int i = 0; i + 1 < W - 1; ++i) hist[i][e] = hist[i + 1][e];
    if (W > 1) hist[W > 1 ? W - 2 : 0][e] = now[e];
  }
  RawV<E, V> out;
  out.put(z);
  return out;
}

// one token each: sequence n is token n; U sequences at a time
template <typename E, int W, int U>
__global__ void __launch_bounds__(CS_THREADS1) conv_token_kernel(const ConvStepArgs a) {
  chain_kernel();
  constexpr int V = CS_VEC1, H = W > 1 ? W - 1 : 1;
  const int c0 = (blockIdx.x * CS_THREADS1 + threadIdx.x) * V;
  if (c0 >= a.C) return;
  const E* x = static_cast<const E*>(a.x) + c0;
  E* y = static_cast<E*>(a.y) + c0;
  E* win = static_cast<E*>(a.window) + c0;
  const int64_t win_slot = (int64_t)(W - 1) * a.C;
  Taps<W, V> k;
  bool first = true;
  for (int n0 = blockIdx.y * U; n0 < a.N; n0 += gridDim.y * U) {
    int from[U], to[U];
    RawV<E, V> row[U], old[U][H];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + u;
      from[u] = to[u] = -2;   // past the last sequence: nothing to do
      if (n >= a.N) continue;
      from[u] = a.slot_in ? a.slot_in[n] : n;
      to[u] = a.slot_out ? a.slot_out[n] : from[u];
      row[u].load(x + (int64_t)n * a.xs);
    }
    if (first) k.load(a, c0);
    first = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool some = from[u] >= 0 && from[u] < a.slots;
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        if (some) old[u][i].load(win + from[u] * win_slot + (int64_t)i * a.C);
        else old[u][i].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + u;
      if (n >= a.N) break;
      if (from[u] < -1 || from[u] >= a.slots) {
        *a.err = ST_DEVICE;
        continue;
      }
      float2 hist[H][V / 2];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) as_pairs(old[u][i], hist[i]);
      conv_row<E, W, V>(k, row[u], hist).store(y + (int64_t)n * a.ys);
      if (to[u] < -1 || to[u] >= a.slots) {
        *a.err = ST_DEVICE;
      } else if (W > 1 && to[u] >= 0) {
        E* p = win + to[u] * win_slot;
#pragma unroll
        for (int i = 0; i + 1 < W - 1; ++i) old[u][i + 1].store(p + (int64_t)i * a.C);
        row[u].store(p + (int64_t)(W - 2) * a.C);
      }
    }
  }
}

// A short sequence: a thread takes CS_FEW tokens at a time, their rows and slots requested together.
template <typename E, int W> __device__ __forceinline__ void short_sequence(const ConvStepArgs& a, int n, int c0) {
  constexpr int V = CS_VEC, H = W - 1;
  const E* x = static_cast<const E*>(a.x) + c0;
  E* y = static_cast<E*>(a.y) + c0;
  E* win = static_cast<E*>(a.window) + c0;
  const int64_t win_slot = (int64_t)H * a.C;
  const int t0 = a.cu[n], t1 = a.cu[n + 1], from = a.slot_in ? a.slot_in[n] : n;
  Taps<W, V> k;
  k.load(a, c0);
  if (t0 < 0 || t1 < t0 || t1 > a.T) {
    *a.err = ST_DEVICE;
    return;
  }
  if (t0 == t1 || t1 - t0 > CS_SHORT) return;
  if (from < -1 || from >= a.slots) {
    *a.err = ST_DEVICE;
    return;
  }
  RawV<E, V> row[H + CS_FEW];   // the rows before the first token, and the tokens'
  float2 hist[W > 1 ? H : 1][V / 2];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    if (from >= 0) row[i].load(win + from * win_slot + (int64_t)i * a.C);
    else row[i].zero();
  }
  for (int t = t0; t < t1; t += CS_FEW) {
    int to[CS_FEW];
#pragma unroll
    for (int i = 0; i < CS_FEW; ++i) {
      to[i] = -1;
      if (t + i >= t1) continue;
      row[H + i].load(x + (int64_t)(t + i) * a.xs);
      to[i] = a.slot_out ? a.slot_out[t + i] : t + i == t1 - 1 ? from : -1;
    }
    if (t == t0) {
#pragma unroll
      for (int i = 0; i < H; ++i) as_pairs(row[i], hist[i]);
    }
#pragma unroll
    for (int i = 0; i < CS_FEW; ++i) {
      if (t + i >= t1) break;
      conv_row<E, W, V>(k, row[H + i], hist).store(y + (int64_t)(t + i) * a.ys);
      if (to[i] == -1) continue;
      if (to[i] < -1 || to[i] >= a.slots) {
        *a.err = ST_DEVICE;
        continue;
      }
#pragma unroll
      for (int j = 0; j < H; ++j) row[i + 1 + j].store(win + to[i] * win_slot + (int64_t)j * a.C);
    }
#pragma unroll
    for (int i = 0; i < H; ++i) row[i] = row[CS_FEW + i];
  }
}

// MIXED: many sequences with few tokens on average.  The first a.N rows of CTAs take a sequence each if it is
// short, the others ranges of tokens, of which they leave those out. (The ranges first: 64 sequences of 8 tokens 8.9 us
// for 8.2, but 63 of one token and one of 400 7.7 for 9.5.)
template <typename E, int W, bool MIXED>
__global__ void __launch_bounds__(CS_THREADS, !MIXED ? 0 : sizeof(E) == 2 ? 6 : 4) conv_step_kernel(const ConvStepArgs a) {
  chain_kernel();
  constexpr int V = CS_VEC, H = W > 1 ? W - 1 : 1, BYTES = V * (int)sizeof(E);
  if (MIXED && blockIdx.y < a.N) {
    const int c = (blockIdx.x * CS_THREADS + threadIdx.x) * V;
    if (c < a.C) short_sequence<E, W>(a, blockIdx.y, c);
    return;
  }
  __shared__ __align__(16) uint8_t ring[CS_STAGES][CS_THREADS * BYTES];
  const int lane = threadIdx.x & 31;
  const int ch = (blockIdx.x * CS_THREADS + threadIdx.x) * V;
  const int c0 = min(ch, a.C - V);   // (threads past the last channel stay for the warps' votes, and store nothing)
  const bool live = ch < a.C;
  const int lo = (blockIdx.y - (MIXED ? a.N : 0)) * a.R, hi = min(lo + a.R, a.T);
  const E* x = static_cast<const E*>(a.x) + c0;
  E* y = static_cast<E*>(a.y) + c0;
  E* win = static_cast<E*>(a.window) + c0;
  const int64_t win_slot = (int64_t)(W - 1) * a.C;
  Taps<W, V> k;
  k.load(a, c0);
  int n = sequence_of(a.cu, a.N, lo);
  // the next sequence from m on that begins before hi and is not short
  auto next_long = [&](int m) {
    for (; m < a.N; m += 32) {
      const bool in = m + lane < a.N;
      const int s = in ? a.cu[m + lane] : 0, e = in ? a.cu[m + lane + 1] : 0;
      const unsigned past = __ballot_sync(~0u, !in || s >= hi);
      const unsigned found = __ballot_sync(~0u, in && s < hi && e > s + CS_SHORT) & (past ? (past & -past) - 1 : ~0u);
      if (found) return m + __ffs(found) - 1;
      if (past) break;
    }
    return a.N;
  };

  // sequence n's tokens [t0, t1); one with bad bounds has none
  int t0, t1, from;
  bool skip;   // the sequence is refused
  auto enter = [&] {
    t0 = a.cu[n];
    t1 = a.cu[n + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.T) t1 = t0;   // (reported apart)
    from = a.slot_in ? a.slot_in[n] : n;
    skip = from < -1 || from >= a.slots;
    if (skip && t0 < t1) *a.err = ST_DEVICE;
  };
  enter();
  // The rows come in order from the first token on, whoever's they are; the last may be the first W-1
  // tokens of a sequence that begins at the range's end.
  if (MIXED && t1 - t0 <= CS_SHORT) {   // (its CTA has reported what is wrong with it)
    if (t0 < lo && t1 >= hi) return;
    n = next_long(n);
    if (n == a.N) return;
    enter();
  }
  int t = t0 < lo ? max(lo, min(t0 + W - 1, t1)) : MIXED ? max(t0, lo) : lo;
  const int stop = min(hi + W - 1, a.T);
  const uint32_t landing = (uint32_t)__cvta_generic_to_shared(&ring[0][threadIdx.x * BYTES]);
  const E* px = x + (int64_t)t * a.xs;
  E* py = y + (int64_t)t * a.ys;
  int fed = t, fill = 0, use = 0;
  auto request = [&] {
    if (fed < stop) {
      if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(landing + fill), "l"(px) : "memory");
      else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(landing + fill), "l"(px) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++fed;
    px += a.xs;
    fill = (fill + CS_THREADS * BYTES) & (CS_STAGES * CS_THREADS * BYTES - 1);
  };
#pragma unroll
  for (int i = 0; i < CS_STAGES - 1; ++i) request();
  // A range meets only the sequences that its tokens lie in, and bad bounds have none: all are looked over here.
  if (!MIXED && blockIdx.x == 0) {
    for (unsigned m = blockIdx.y * CS_THREADS + threadIdx.x; m < (unsigned)a.N; m += gridDim.y * CS_THREADS) {
      const int b = a.cu[m], e = a.cu[m + 1];
      if (b < 0 || e < b || e > a.T) *a.err = ST_DEVICE;
    }
  }
  // the row of token t, which is then passed
  auto take = [&](RawV<E, V>* row) {
    asm volatile("cp.async.wait_group %0;" ::"n"(CS_STAGES - 2) : "memory");
    row->load_shared(landing + use);
    use = (use + CS_THREADS * BYTES) & (CS_STAGES * CS_THREADS * BYTES - 1);
    request();   // into the slot before
    ++t;
    py += a.ys;
  };
  float2 hist[H][V / 2];
  // up to `end` of the sequence; hist holds the rows before
  auto walk = [&](const int end) {
    auto one = [&] {
      E* out = py;
      RawV<E, V> row;
      take(&row);
      const RawV<E, V> r = conv_row<E, W, V>(k, row, hist);
      if (live) r.store(out);
    };
    for (; t + 4 <= end;) {   // (four at a time the rows of hist change names, not registers)
      one();
      one();
      one();
      one();
    }
    while (t < end) one();
  };

  if (t0 < lo) {   // a sequence that began in an earlier range; its tokens before t are the first token's CTA's
    const int end = min(t1, hi);
    if (t < end && !skip) {
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        RawV<E, V> r;
        r.load(x + (int64_t)(t - (W - 1) + i) * a.xs);
        as_pairs(r, hist[i]);
      }
      walk(end);
    }
    if (t1 >= hi) return;
    ++n;
  }
  if (MIXED) n = next_long(n);
  for (; n < a.N; n = MIXED ? next_long(n + 1) : n + 1) {   // the sequences that begin in this range
    enter();
    if (t0 >= hi) return;
    if (t0 == t1 || t0 < lo || skip) continue;
    RawV<E, V> old[H], passed;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      if (from >= 0) old[i].load(win + from * win_slot + (int64_t)i * a.C);
      else old[i].zero();
      as_pairs(old[i], hist[i]);
    }
    while (t < t0) take(&passed);   // the tokens of sequences that were refused
    walk(min(t1, max(hi, t0 + W - 1)));
    // the windows of the sequence's tokens, looked up CS_LOOK * 32 at a time
    for (int s0 = a.slot_out ? t0 : t1 - 1; s0 < t1; s0 += CS_LOOK * 32) {
      int to[CS_LOOK];
#pragma unroll
      for (int q = 0; q < CS_LOOK; ++q) {
        const int s = s0 + q * 32 + lane;
        to[q] = s >= t1 ? -1 : a.slot_out ? a.slot_out[s] : q + lane == 0 ? from : -1;
      }
#pragma unroll
      for (int q = 0; q < CS_LOOK; ++q) {
        if (to[q] < -1 || to[q] >= a.slots) *a.err = ST_DEVICE;
        for (unsigned hits = W > 1 ? __ballot_sync(~0u, to[q] >= 0 && to[q] < a.slots) : 0u; hits; hits &= hits - 1) {
          const int i0 = __ffs(hits) - 1, first = s0 + q * 32 + i0 - t0 - (W - 2);
          E* p = win + __shfl_sync(~0u, to[q], i0) * win_slot;
#pragma unroll
          for (int i = 0; i < W - 1; ++i) {
            const int back = first + i;   // the row's place in the sequence; before it: the old window's
            RawV<E, V> r;
            if (back >= 0) r.load(x + (int64_t)(t0 + back) * a.xs);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
              if (back + W - 1 == j) r = old[j];
            if (live) r.store(p + (int64_t)i * a.C);
          }
        }
      }
    }
    if (t1 >= hi) return;
  }
}

template <typename E, int W> static void launch_conv_step(const ConvStepArgs& a, bool mixed, dim3 grid, cudaStream_t s) {
  if (a.cu && mixed) launch_chained(conv_step_kernel<E, W, true>, grid, CS_THREADS, 0, s, a);
  else if (a.cu) launch_chained(conv_step_kernel<E, W, false>, grid, CS_THREADS, 0, s, a);
  else if (a.R == 1) launch_chained(conv_token_kernel<E, W, 1>, grid, CS_THREADS1, 0, s, a);
  else launch_chained(conv_token_kernel<E, W, 2>, grid, CS_THREADS1, 0, s, a);
}
template <typename E> static void launch_conv_step(const ConvStepArgs& a, int W, bool mixed, dim3 grid, cudaStream_t s) {
  switch (W) {
    case 1: launch_conv_step<E, 1>(a, mixed, grid, s); break;
    case 2: launch_conv_step<E, 2>(a, mixed, grid, s); break;
    case 3: launch_conv_step<E, 3>(a, mixed, grid, s); break;
    default: launch_conv_step<E, 4>(a, mixed, grid, s); break;
  }
}

static bool conv_stride(int64_t* s, int C, int esize) {
  if (*s == 0) *s = C;
  return *s >= C && *s * esize % 16 == 0;
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_conv1d_step(const gdn_conv_step_problem* p, const void* x, const float* w, const float* b,
                                      const int32_t* cu_dev, const int32_t* slot_in, const int32_t* slot_out,
                                      void* window, void* y, int32_t* dev_err, struct CUstream_st* stream) {
  if (!p || p->T < 0 || p->N < 0 || p->C < 8 || p->C % 8 != 0 || p->W < 1 || p->slots < 0) return GDN_ERR_INVALID_ARG;
  if (p->W > 4 || p->T > (int64_t)INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (!cu_dev && p->T != p->N) return GDN_ERR_INVALID_ARG;
  if (!slot_in && p->slots < p->N) return GDN_ERR_INVALID_ARG;
  ConvStepArgs a;
  a.xs = p->x_stride;
  a.ys = p->y_stride;
  const int es = elem_bytes(p->dtype);
  if (!conv_stride(&a.xs, p->C, es) || !conv_stride(&a.ys, p->C, es)) return GDN_ERR_INVALID_ARG;
  if (!dev_err) return GDN_ERR_INVALID_ARG;
  if (p->T == 0 || p->N == 0) return GDN_OK;
  if (!aligned16(x) || !aligned16(y) || !aligned16(w) || (b && !aligned16(b)) ||
      (p->W > 1 && p->slots > 0 && !aligned16(window)) || !on_words(cu_dev, slot_in, slot_out, dev_err))
    return GDN_ERR_INVALID_ARG;
  a.x = x;
  a.w = w;
  a.b = b;
  a.cu = cu_dev;
  a.slot_in = slot_in;
  a.slot_out = slot_out;
  a.window = window;
  a.y = y;
  a.err = dev_err;
  a.T = (int)p->T;
  a.N = p->N;
  a.C = p->C;
  a.slots = p->slots;
  const int per_cta = cu_dev ? CS_THREADS * CS_VEC : CS_THREADS1 * CS_VEC1;
  const int cols = (p->C + per_cta - 1) / per_cta;
  // Few tokens a sequence on average: short sequences apart from the ranges (10,240 channels, 64 of 1-4 tokens: 5.8 us against
  // 8.6; 63 of one and one of 400: 9.5 against 19.0; 64 of 8: 8.2 against 10.1; but 256 of 8: 26.2 against 26.3, 256 of
  // 16: 46 against 45, 64 of 20: 17 against 14).  32,768 of them and the ranges of their tokens fit grid.y.
  const bool mixed = cu_dev && p->N <= 32768 && p->T <= (int64_t)p->N * CS_MEAN;
  int64_t rows;
  if (cu_dev) {
    // one round of CTAs, whose start is most of their time while ranges are short, or several of longer ones (29
    // sequences of up to 106 tokens: one round of 24 tokens 14 us, four of 6 23 us)
    const int64_t round = std::max<int64_t>(1, (int64_t)sm_count() * CS_ROUND / cols), one = (p->T + round - 1) / round;
    a.R = (int)(one <= CS_LONG ? one : std::min<int64_t>(CS_MAXR, std::max<int64_t>(CS_LONG, (one + 3) / 4)));
    if (mixed) a.R = std::max(a.R, CS_SHORT);   // (262,144 tokens at most: no more rows than the grid has)
    else a.R = std::max(a.R, (int)((p->T + CS_ROWS - 1) / CS_ROWS));
    rows = (p->T + a.R - 1) / a.R + (mixed ? p->N : 0);
  } else {
    // one sequence a CTA column while the GPU holds them all, then two (BF16, 10,240 channels, in a graph: 64 3.17 us
    // with one, 3.07 with two; 512 13.1 and 13.4), side by side as far as they give an SM 32 CTAs
    a.R = (int64_t)p->N * cols <= (int64_t)sm_count() * CS_ROUND1 * 128 / CS_THREADS1 ? 1 : 2;
    rows = std::min<int64_t>((p->N + a.R - 1) / a.R, std::max<int64_t>(1, (int64_t)sm_count() * 32 / cols));
  }
  const dim3 grid(cols, (unsigned)rows);
  prof_begin(K_CONV_STEP, stream);
  switch (p->dtype) {
    case GDN_BF16: launch_conv_step<__nv_bfloat16>(a, p->W, mixed, grid, stream); break;
    case GDN_FP16: launch_conv_step<__half>(a, p->W, mixed, grid, stream); break;
    default: launch_conv_step<float>(a, p->W, mixed, grid, stream); break;
  }
  prof_end(K_CONV_STEP, stream);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
