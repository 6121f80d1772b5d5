// gdn_conv_step.cu -- the causal convolution + SiLU on a pool of windows, for generation: the
// next tokens of N sequences, the last W-1 rows of each kept in its slot.
//   z[t, c] = b[c] + sum_i w[c, i] row(t - (W-1) + i)[c],  y = z sigma(z)
// with row(s) the token s of the sequence, or its window's row before the first token.
//
// A thread owns 8 channels and walks a range of tokens with the last W-1 rows in registers.  Long
// sequences are cut over CTAs; a slot may be read and written by the same call, so whatever reads
// or writes a sequence's slots is done by one CTA, the one whose range holds the sequence's first
// token: it also computes the W-1 tokens at the start that need the window (past its range's end if
// they lie there), and writes the windows of all the sequence's tokens, each thread after it has read the old
// window of its channels.
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_prof.h"

namespace gdn {

constexpr int CS_THREADS = 128;
constexpr int CS_VEC = 8;         // channels per thread
constexpr int CS_BATCH = 4;       // rows requested together
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

template <typename E, int W>
__global__ void __launch_bounds__(CS_THREADS) conv_step_kernel(const ConvStepArgs a) {
  constexpr int H = W > 1 ? W - 1 : 1;
  const int c0 = (blockIdx.x * CS_THREADS + threadIdx.x) * CS_VEC;
  const int lo = blockIdx.y * a.R, hi = min(lo + a.R, a.T);
  int n = a.cu ? sequence_of(a.cu, a.N, lo) : lo;
  if (c0 >= a.C) return;   // (whole threads; the warps' search is done)
  float w[W][CS_VEC], b[CS_VEC];
#pragma unroll
  for (int e = 0; e < CS_VEC; ++e) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i][e] = a.w[(int64_t)(c0 + e) * W + i];
    b[e] = a.b ? a.b[c0 + e] : 0.f;
  }
  const E* x = static_cast<const E*>(a.x) + c0;
  E* y = static_cast<E*>(a.y) + c0;
  E* win = static_cast<E*>(a.window) + c0;
  const int64_t win_slot = (int64_t)(W - 1) * a.C;
  Raw8<E> hist[H];   // the W-1 rows before the next token, the newest last

  // sequence n's tokens [t0, t1); one with bad bounds has none
  int t0, t1, from;
  bool mine, skip;   // this CTA serves the sequence's slots; the sequence is refused
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
  // tokens [t, end) of the sequence; hist holds the rows before t
  auto walk = [&](int t, const int end) {
    for (; t < end; t += CS_BATCH) {
      Raw8<E> row[CS_BATCH];
#pragma unroll
      for (int u = 0; u < CS_BATCH; ++u)
        if (t + u < end) row[u].load(x + (int64_t)(t + u) * a.xs);
#pragma unroll
      for (int u = 0; u < CS_BATCH; ++u) {
        if (t + u >= end) break;
        float z[CS_VEC], f[CS_VEC];
#pragma unroll
        for (int e = 0; e < CS_VEC; ++e) z[e] = b[e];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          hist[i].get(f);
#pragma unroll
          for (int e = 0; e < CS_VEC; ++e) z[e] = fmaf(w[i][e], f[e], z[e]);
        }
        row[u].get(f);
#pragma unroll
        for (int e = 0; e < CS_VEC; ++e) {
          z[e] = fmaf(w[W - 1][e], f[e], z[e]);
          z[e] = z[e] / (1.f + expf(-z[e]));
        }
        Raw8<E> out;
        out.put(z);
        out.store(y + (int64_t)(t + u) * a.ys);
        if (W > 1) {
#pragma unroll
          for (int i = 0; i + 1 < W - 1; ++i) hist[i] = hist[i + 1];
          hist[H - 1] = row[u];
          if (mine) {
            const int to = a.slot_out ? a.slot_out[t + u] : t + u == t1 - 1 ? from : -1;
            if (to < -1 || to >= a.slots) {
              *a.err = ST_DEVICE;
            } else if (to >= 0) {
#pragma unroll
              for (int i = 0; i < W - 1; ++i) hist[i].store(win + to * win_slot + (int64_t)i * a.C);
            }
          }
        }
      }
    }
  };

  enter();
  if (t0 < lo) {   // a sequence that began in an earlier range
    mine = false;
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
    mine = true;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      if (from >= 0) hist[i].load(win + from * win_slot + (int64_t)i * a.C);
      else hist[i].zero();
    }
    const int end = min(t1, max(hi, t0 + W - 1));
    walk(t0, end);
    if (W > 1 && end < t1) {   // the other tokens are other CTAs', but the windows are this one's
      for (int s = a.slot_out ? end : t1 - 1; s < t1; ++s) {
        const int to = a.slot_out ? a.slot_out[s] : from;
        if (to < -1 || to >= a.slots) *a.err = ST_DEVICE;
        if (to < 0 || to >= a.slots) continue;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {   // (s >= t0 + W - 1: all of them are tokens)
          Raw8<E> r;
          r.load(x + (int64_t)(s - (W - 2) + i) * a.xs);
          r.store(win + to * win_slot + (int64_t)i * a.C);
        }
      }
    }
    if (t1 >= hi) return;
  }
}

template <typename E>
static void launch_conv_step(const ConvStepArgs& a, int W, dim3 grid, cudaStream_t s) {
  switch (W) {
    case 1: conv_step_kernel<E, 1><<<grid, CS_THREADS, 0, s>>>(a); break;
    case 2: conv_step_kernel<E, 2><<<grid, CS_THREADS, 0, s>>>(a); break;
    case 3: conv_step_kernel<E, 3><<<grid, CS_THREADS, 0, s>>>(a); break;
    default: conv_step_kernel<E, 4><<<grid, CS_THREADS, 0, s>>>(a); break;
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
  // one token per CTA while that leaves the GPU idle, then longer ranges, which read the taps less often
  const int cols = (p->C + CS_THREADS * CS_VEC - 1) / (CS_THREADS * CS_VEC);
  const int64_t ranges = std::max<int64_t>(1, (int64_t)sm_count() * 16 / cols);
  a.R = (int)std::min<int64_t>(CS_MAXR, (p->T + ranges - 1) / ranges);
  const int64_t rows = (p->T + a.R - 1) / a.R;
  const dim3 grid(cols, (unsigned)rows);
  if (rows > 65535) return GDN_ERR_UNSUPPORTED;   // grid.y: more than 4 M tokens
  prof_begin(K_CONV_STEP, stream);
  switch (p->dtype) {
    case GDN_BF16: launch_conv_step<__nv_bfloat16>(a, p->W, grid, stream); break;
    case GDN_FP16: launch_conv_step<__half>(a, p->W, grid, stream); break;
    default: launch_conv_step<float>(a, p->W, grid, stream); break;
  }
  prof_end(K_CONV_STEP, stream);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
