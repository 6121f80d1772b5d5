// gdn_conv_step.cu -- the causal convolution + SiLU on a pool of windows, for generation: the
// next tokens of N sequences, the last W-1 rows of each kept in its slot.
//   z[t, c] = b[c] + sum_i w[c, i] row(t - (W-1) + i)[c],  y = z sigma(z)
// with row(s) the token s of the sequence, or its window's row before the first token.
//
// Bandwidth-bound: a thread owns V neighbouring channels and walks a range of tokens with the last W-1 rows in
// registers, CS_BATCH rows requested at a time. Few tokens: V = 2 and a range of one token, for the most
// threads and the shortest chain of loads (64 single tokens of 10,240 channels: TIME_SMALL). Many: V = 4 and ranges
// of up to 64, which read the taps less often (28,800 tokens: TIME_LARGE).
//
// Long sequences are cut over CTAs, and a slot may be read and written by the same call, so whatever
// reads or writes a sequence's slots is done by one CTA per channel block, the one whose range holds its first
// token: it also computes the first W-1 tokens, which need the window (past its range's end if they lie
// there), and writes the windows of all the sequence's tokens from its own copy of the old window and x.
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_prof.h"

namespace gdn {

constexpr int CS_THREADS = 128;
constexpr int CS_BATCH = 8;       // rows requested together
constexpr int CS_MAXR = 64;       // tokens per range, at most

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
  int T, N, C, slots, R;
};

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

template <typename E, int W, int V>
__global__ void __launch_bounds__(CS_THREADS) conv_step_kernel(const ConvStepArgs a) {
  constexpr int H = W > 1 ? W - 1 : 1;
  const int lane = threadIdx.x & 31;
  const int ch = (blockIdx.x * CS_THREADS + threadIdx.x) * V;
  const int c0 = min(ch, a.C - V);   // (threads past the last channel stay for the warps' votes, and store nothing)
  const bool live = ch < a.C;
  const int lo = blockIdx.y * a.R, hi = min(lo + a.R, a.T);
  const E* x = static_cast<const E*>(a.x) + c0;
  E* y = static_cast<E*>(a.y) + c0;
  E* win = static_cast<E*>(a.window) + c0;
  const int64_t win_slot = (int64_t)(W - 1) * a.C;
  float w[V][W], b[V];
  {
    RawV<float, 4> taps[V * W / 4 > 0 ? V * W / 4 : 1];
    const float* wp = a.w + (int64_t)c0 * W;
    if constexpr (V * W % 4 == 0) {   // (c0 is a multiple of V: 16-byte aligned)
#pragma unroll
      for (int i = 0; i < V * W / 4; ++i) {
        taps[i].load(wp + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[(4 * i + j) / W][(4 * i + j) % W] = __uint_as_float(taps[i].u[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V * W; ++i) w[i / W][i % W] = wp[i];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) b[e] = a.b ? a.b[c0 + e] : 0.f;
  }
  int n = a.cu ? sequence_of(a.cu, a.N, lo) : lo;

  // sequence n's tokens [t0, t1); one with bad bounds has none
  int t0, t1, from;
  bool skip;   // the sequence is refused
  auto enter = [&] {
    t0 = a.cu ? a.cu[n] : n;
    t1 = a.cu ? a.cu[n + 1] : n + 1;
    if (t0 < 0 || t1 < t0 || t1 > a.T) {
      *a.err = ST_DEVICE;
      t1 = t0;
    }
    from = a.slot_in ? a.slot_in[n] : n;
    skip = from < -1 || from >= a.slots;
    if (skip && t0 < t1) *a.err = ST_DEVICE;
  };
  RawV<E, V> hist[H];   // the W-1 rows before the next token, the newest last
  // tokens [t, end) of the sequence; hist holds the rows before t
  auto walk = [&](int t, const int end) {
    for (; t < end; t += CS_BATCH) {
      RawV<E, V> row[CS_BATCH];
#pragma unroll
      for (int u = 0; u < CS_BATCH; ++u)
        if (t + u < end) row[u].load(x + (int64_t)(t + u) * a.xs);
#pragma unroll
      for (int u = 0; u < CS_BATCH; ++u) {
        if (t + u >= end) break;
        float z[V], f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] = b[e];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          if (i < W - 1) hist[i].get(f);
          else row[u].get(f);
#pragma unroll
          for (int e = 0; e < V; ++e) z[e] = fmaf(w[e][i], f[e], z[e]);
        }
        // the fast exponential and division: a few last places, in a value that is rounded to E
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] = __fdividef(z[e], 1.f + __expf(-z[e]));
        RawV<E, V> out;
        out.put(z);
        if (live) out.store(y + (int64_t)(t + u) * a.ys);
#pragma unroll
        for (int i = 0; i + 1 < W - 1; ++i) hist[i] = hist[i + 1];
        if (W > 1) hist[H - 1] = row[u];
      }
    }
  };

  enter();
  if (t0 < lo) {   // a sequence that began in an earlier range
    const int t = max(lo, min(t0 + W - 1, t1));   // the tokens before are the first token's CTA's
    const int end = min(t1, hi);
    if (t < end && !skip) {
#pragma unroll
      for (int i = 0; i < W - 1; ++i) hist[i].load(x + (int64_t)(t - (W - 1) + i) * a.xs);
      walk(t, end);
    }
    if (t1 >= hi) return;
    ++n;
  }
  for (; n < a.N; ++n) {   // the sequences that begin in this range
    enter();
    if (t0 >= hi) return;
    if (t0 == t1 || t0 < lo || skip) continue;
    RawV<E, V> old[H];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      if (from >= 0) old[i].load(win + from * win_slot + (int64_t)i * a.C);
      else old[i].zero();
      hist[i] = old[i];
    }
    walk(t0, min(t1, max(hi, t0 + W - 1)));
    if (W > 1) {
      // the windows of the sequence's tokens: 32 of them are looked up at a time
      for (int s0 = a.slot_out ? t0 : t1 - 1; s0 < t1; s0 += 32) {
        const int to = s0 + lane >= t1 ? -1 : a.slot_out ? a.slot_out[s0 + lane] : lane == 0 ? from : -1;
        if (to < -1 || to >= a.slots) *a.err = ST_DEVICE;
        for (unsigned hits = __ballot_sync(~0u, to >= 0 && to < a.slots); hits; hits &= hits - 1) {
          const int i0 = __ffs(hits) - 1, s = s0 + i0;
          E* p = win + __shfl_sync(~0u, to, i0) * win_slot;
#pragma unroll
          for (int i = 0; i < W - 1; ++i) {
            const int back = s - t0 - (W - 2) + i;   // the row's place in the sequence; before it: the old window's
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

template <typename E, int V>
static void launch_conv_step(const ConvStepArgs& a, int W, dim3 grid, cudaStream_t s) {
  switch (W) {
    case 1: conv_step_kernel<E, 1, V><<<grid, CS_THREADS, 0, s>>>(a); break;
    case 2: conv_step_kernel<E, 2, V><<<grid, CS_THREADS, 0, s>>>(a); break;
    case 3: conv_step_kernel<E, 3, V><<<grid, CS_THREADS, 0, s>>>(a); break;
    default: conv_step_kernel<E, 4, V><<<grid, CS_THREADS, 0, s>>>(a); break;
  }
}
template <typename E>
static void launch_conv_step(const ConvStepArgs& a, int W, int vec, dim3 grid, cudaStream_t s) {
  if (vec == 2) launch_conv_step<E, 2>(a, W, grid, s);
  else launch_conv_step<E, 4>(a, W, grid, s);
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
      (p->W > 1 && p->slots > 0 && !aligned16(window)))
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
  // few tokens: two channels a thread and a token a CTA; many: four channels, and ranges that leave every
  // SM 16 CTAs
  const bool few = p->T * p->C < (int64_t)sm_count() * 4096;
  const int vec = few ? 2 : 4;
  const int cols = (p->C + CS_THREADS * vec - 1) / (CS_THREADS * vec);
  const int64_t ranges = std::max<int64_t>(1, (int64_t)sm_count() * 16 / cols);
  a.R = few ? 1 : (int)std::min<int64_t>(CS_MAXR, (p->T + ranges - 1) / ranges);
  const int64_t rows = (p->T + a.R - 1) / a.R;
  if (rows > 65535) return GDN_ERR_UNSUPPORTED;   // grid.y: 4 M tokens, or fewer in very many columns
  const dim3 grid(cols, (unsigned)rows);
  prof_begin(K_CONV_STEP, stream);
  switch (p->dtype) {
    case GDN_BF16: launch_conv_step<__nv_bfloat16>(a, p->W, vec, grid, stream); break;
    case GDN_FP16: launch_conv_step<__half>(a, p->W, vec, grid, stream); break;
    default: launch_conv_step<float>(a, p->W, vec, grid, stream); break;
  }
  prof_end(K_CONV_STEP, stream);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
