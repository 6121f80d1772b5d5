// gdn_norm.cu -- the root-mean-square norm of the residual stream, with the addition in front of it, an output in 8 bits
// beside the one in the input's type, and its gradients.
//
//   h = x + r (rounded to the type, and it is the rounded value that goes on),  z = h rho w,  rho = 1 / sqrt(mean h^2 + eps)
//   s = max |z| / 448 over a row or group,  z8 = e4m3(z / s)
//   dh = rho (g - h rho^2 mean(g h)) + (what arrives along the stream),  g = dz w;   dw = sum over the rows of dz h rho
//
// Bound by the bytes: each row is read once and stays in registers (8 values a thread at a time, VPT such pieces) while its
// sums go round.  Short rows belong to a warp, longer ones to a CTA.  65,536 rows of 4,096 BF16 values, both outputs: 375 us, 95%
// of a plain copy's rate; backward 333 us, 95%.
#include <cuda_runtime.h>

#include <type_traits>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_prof.h"

namespace gdn {

constexpr float NORM_E4M3 = 448.f;               // the largest value of the 8-bit type
constexpr float NORM_LEAST = 0x1p-100f;          // the least scale: rows of zeros have one, too
constexpr int NORM_GENERAL = 256;                // threads of the kernels for rows of any kind

struct NormArgs {
  const void* x;      // backward: h
  const void* r;      // or null; backward: what arrives along the stream
  const void* dy;     // backward
  const float* w;
  void* h;            // or null
  void* y;            // or null; backward: dx
  uint8_t* y8;        // or null
  float* scales;
  float* partial;     // backward: [CTAs][C], or null: no dw
  int64_t T, xs, rs, hs, ys;   // backward: xs of h, rs of what arrives, hs of dy, ys of dx
  int C, group;
  float eps;
};

__device__ __forceinline__ uint16_t e4m3_pair(float lo, float hi) {
  uint16_t u;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(hi), "f"(lo));
  return u;
}
__device__ __forceinline__ float norm_inverse(float ss, int C, float eps) { return 1.f / sqrtf(ss / (float)C + eps); }

// sums (or the larger) over a row's threads: a warp, or the CTA with one word of shared memory a warp
template <bool MAX> __device__ __forceinline__ float over_warp(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float o = __shfl_xor_sync(~0u, v, d);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  return v;
}
template <bool MAX> __device__ __forceinline__ float over_row(float v, bool one_warp, float* words) {
  v = over_warp<MAX>(v);
  if (one_warp) return v;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) words[threadIdx.x >> 5] = v;
  __syncthreads();
  return over_warp<MAX>(lane < warps ? words[lane] : 0.f);   // (all that is summed or compared is 0 or more, or a sum)
}

template <typename E, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : VPT * sizeof(E) <= 4 ? 1024 : 512) norm_fwd_kernel(const NormArgs a) {
  chain_kernel();
  __shared__ float words[2][32];
  const int pieces = a.C >> 3, step = WARP ? 32 : blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t rows = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  Raw8<E> nx[VPT], nr[VPT];
  auto request = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int p = me + i * step;
      if (p < pieces && row < a.T) {
        nx[i].load(static_cast<const E*>(a.x) + row * a.xs + p * 8);
        if (a.r) nr[i].load(static_cast<const E*>(a.r) + row * a.rs + p * 8);
      }
    }
  };
  request(t);
  for (; t < a.T; t += rows) {
    float v[VPT][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int p = me + i * step;
      if (p < pieces) {
        nx[i].get(v[i]);
        if (a.r) {
          float u[8];
          nr[i].get(u);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += u[j];
          Raw8<E> out;
          out.put(v[i]);
          out.store(static_cast<E*>(a.h) + t * a.hs + p * 8);
          out.get(v[i]);
        } else if (a.h) {
          nx[i].store(static_cast<E*>(a.h) + t * a.hs + p * 8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
      }
    }
    request(t + rows);
    const float rho = norm_inverse(over_row<false>(ss, WARP, words[0]), a.C, a.eps);
    float most[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int p = me + i * step;
      most[i] = 0.f;
      if (p < pieces) {
        const float4 w0 = reinterpret_cast<const float4*>(a.w + p * 8)[0], w1 = reinterpret_cast<const float4*>(a.w + p * 8)[1];
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = v[i][j] * rho * w[j];
          most[i] = fmaxf(most[i], fabsf(v[i][j]));
        }
        if (a.y) {
          Raw8<E> out;
          out.put(v[i]);
          out.store(static_cast<E*>(a.y) + t * a.ys + p * 8);
        }
      }
    }
    if (!a.y8) continue;
    if (a.group == a.C) {
      float m = most[0];
#pragma unroll
      for (int i = 1; i < VPT; ++i) m = fmaxf(m, most[i]);
      m = over_row<true>(m, WARP, words[1]);
#pragma unroll
      for (int i = 0; i < VPT; ++i) most[i] = m;
      if (me == 0) a.scales[t] = fmaxf(m, NORM_E4M3 * NORM_LEAST) / NORM_E4M3;
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {   // a group is 4, 8 or 16 neighbouring lanes
        float m = most[i];
        for (int d = 1; d * 8 < a.group; d <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        most[i] = m;
        const int c = (me + i * step) * 8;
        if (c < a.C && c % a.group == 0)
          a.scales[t * (a.C / a.group) + c / a.group] = fmaxf(m, NORM_E4M3 * NORM_LEAST) / NORM_E4M3;
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int p = me + i * step;
      if (p < pieces) {
        const float f = NORM_E4M3 / fmaxf(most[i], NORM_E4M3 * NORM_LEAST);
        uint2 u;
        u.x = e4m3_pair(v[i][0] * f, v[i][1] * f) | (uint32_t)e4m3_pair(v[i][2] * f, v[i][3] * f) << 16;
        u.y = e4m3_pair(v[i][4] * f, v[i][5] * f) | (uint32_t)e4m3_pair(v[i][6] * f, v[i][7] * f) << 16;
        *reinterpret_cast<uint2*>(a.y8 + t * a.C + p * 8) = u;
      }
    }
  }
}

// Rows of a warp, backward: the next is asked for a row ahead, as far as there are registers for it.
template <typename E, int VPT> __global__ void __launch_bounds__(128) norm_bwd_kernel(const NormArgs a) {
  chain_kernel();
  const int pieces = a.C >> 3, step = 32, me = threadIdx.x & 31;
  const int64_t rows = (int64_t)gridDim.x * (blockDim.x >> 5), first = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  constexpr bool AHEAD = VPT * sizeof(E) <= 4;
  Raw8<E> nh[VPT], ng[VPT], na[VPT];
  float dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT * 8; ++i) dw[i >> 3][i & 7] = 0.f;
  auto request = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int p = me + i * step;
      if (p < pieces && row < a.T) {
        nh[i].load(static_cast<const E*>(a.x) + row * a.xs + p * 8);
        ng[i].load(static_cast<const E*>(a.dy) + row * a.hs + p * 8);
        if (AHEAD && a.r) na[i].load(static_cast<const E*>(a.r) + row * a.rs + p * 8);
      }
    }
  };
  if (AHEAD) request(first);
  for (int64_t t = first; t < a.T; t += rows) {
    if (!AHEAD) request(t);
    Raw8<E> h[VPT], g[VPT], along[VPT];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int p = me + i * step;
      h[i] = nh[i], g[i] = ng[i];
      if (AHEAD) along[i] = na[i];
      if (p < pieces) {
        float hv[8], gv[8];
        h[i].get(hv);
        g[i].get(gv);
        const float4 w0 = reinterpret_cast<const float4*>(a.w + p * 8)[0], w1 = reinterpret_cast<const float4*>(a.w + p * 8)[1];
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(hv[j], hv[j], ss);
          sg = fmaf(gv[j] * w[j], hv[j], sg);
        }
      }
    }
    if (AHEAD) request(t + rows);
    ss = over_warp<false>(ss);
    float mean = over_warp<false>(sg);
    const float rho = norm_inverse(ss, a.C, a.eps);
    mean = mean * rho / (float)a.C;   // of g and the normed h
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int p = me + i * step;
      if (p < pieces) {
        float hv[8], gv[8], av[8];
        h[i].get(hv);
        g[i].get(gv);
        if (a.r) {
          if (!AHEAD) along[i].load(static_cast<const E*>(a.r) + t * a.rs + p * 8);
          along[i].get(av);
        }
        const float4 w0 = reinterpret_cast<const float4*>(a.w + p * 8)[0], w1 = reinterpret_cast<const float4*>(a.w + p * 8)[1];
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xhat = hv[j] * rho;
          dw[i][j] = fmaf(gv[j], xhat, dw[i][j]);
          hv[j] = rho * fmaf(-xhat, mean, gv[j] * w[j]) + (a.r ? av[j] : 0.f);
        }
        Raw8<E> out;
        out.put(hv);
        out.store(static_cast<E*>(a.y) + t * a.ys + p * 8);
      }
    }
  }
  if (!a.partial) return;
  // this CTA's part of dw: its warps' one after the other
  extern __shared__ float sums[];   // [warps][C]
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int p = me + i * 32;
    if (p < pieces)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[(threadIdx.x >> 5) * a.C + p * 8 + j] = dw[i][j];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
    float v = 0.f;
    for (int n = 0; n < (int)(blockDim.x >> 5); ++n) v += sums[n * a.C + c];
    a.partial[(int64_t)blockIdx.x * a.C + c] = v;
  }
}

// Rows of a CTA, backward.  The rows ahead are copied to shared memory, so many that an SM's CTAs have some 200 KB on the way,
// and not to registers, so that three CTAs of 256 threads fit (65,536 rows of 4,096 BF16 values 333 us, 95% of a plain copy's
// rate; two 363; with one row ahead in registers 365).  A thread's copies are its own to read: no barrier but for the sums.  Its
// 8 VPT values are words of 16 bytes a whole CTA's width apart: the copies pass the L1, and would fetch sectors twice (30,517
// FP32 rows: 304 us; words in pairs 485; without rows ahead 406).
template <typename E, int VPT> struct NormAhead {
  static constexpr int U = 16 / (int)sizeof(E), N = 8 * VPT / U;   // values of a word, words of a thread's row
  static constexpr int ROWS = N == 2 ? 3 : 8 / N;
  static constexpr int BYTES = ROWS * 3 * N * 16;   // a thread
};
template <typename E> struct NormWord : Raw8<E> {};
template <> struct NormWord<float> {
  float4 u;
  __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w; }
  __device__ __forceinline__ void put(const float (&v)[4]) { u = make_float4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = u; }
};

template <typename E, int VPT> __global__ void __launch_bounds__(512) norm_bwd_rows_kernel(const NormArgs a) {
  chain_kernel();
  using Ahead = NormAhead<E, VPT>;
  constexpr int U = Ahead::U, N = Ahead::N;
  constexpr bool KEEP = VPT <= 2;   // the weights stay in registers
  extern __shared__ uint4 ahead[];
  __shared__ float words[2][32];
  const int all = a.C / U, step = blockDim.x, me = threadIdx.x, lane = me & 31, warps = blockDim.x >> 5;
  const int64_t rows = gridDim.x;
  auto slot = [&](int stage, int stream, int i) { return ahead + ((stage * 3 + stream) * N + i) * step + me; };
  auto request = [&](int stage, int64_t row) {
    if (row < a.T) {
      const E* from[3] = {static_cast<const E*>(a.x) + row * a.xs, static_cast<const E*>(a.dy) + row * a.hs,
                          a.r ? static_cast<const E*>(a.r) + row * a.rs : nullptr};
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (me + i * step < all && from[k])
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot(stage, k, i))),
                         "l"(from[k] + (me + i * step) * U)
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch = [&](int stage, int stream, int i, float (&v)[U]) {
    NormWord<E> x;
    *reinterpret_cast<uint4*>(&x) = *slot(stage, stream, i);
    x.get(v);
  };
  float dw[N][U], kept[KEEP ? N : 1][U];
  auto weights = [&](int i, float (&w)[U]) {
#pragma unroll
    for (int j = 0; j < U; j += 4) {
      const float4 x = *reinterpret_cast<const float4*>(a.w + (me + i * step) * U + j);
      w[j] = x.x, w[j + 1] = x.y, w[j + 2] = x.z, w[j + 3] = x.w;
    }
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < U; ++j) dw[i][j] = 0.f;
    if (KEEP && me + i * step < all) weights(i, kept[KEEP ? i : 0]);
  }
  int64_t t = blockIdx.x;
#pragma unroll
  for (int k = 0; k < Ahead::ROWS; ++k) request(k, t + k * rows);
  for (int stage = 0; t < a.T; t += rows, stage = stage + 1 == Ahead::ROWS ? 0 : stage + 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(Ahead::ROWS - 1) : "memory");
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (me + i * step < all) {
        float h[U], g[U], w[U];
        fetch(stage, 0, i, h);
        fetch(stage, 1, i, g);
        if (!KEEP) weights(i, w);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          ss = fmaf(h[j], h[j], ss);
          sg = fmaf(g[j] * (KEEP ? kept[KEEP ? i : 0][j] : w[j]), h[j], sg);
        }
      }
    }
    ss = over_warp<false>(ss);
    sg = over_warp<false>(sg);
    __syncthreads();
    if (lane == 0) words[0][me >> 5] = ss, words[1][me >> 5] = sg;
    __syncthreads();
    ss = over_warp<false>(lane < warps ? words[0][lane] : 0.f);
    sg = over_warp<false>(lane < warps ? words[1][lane] : 0.f);
    const float rho = norm_inverse(ss, a.C, a.eps), mean = sg * rho / (float)a.C;   // of g and the normed h
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (me + i * step < all) {
        float h[U], g[U], along[U], w[U];
        fetch(stage, 0, i, h);
        fetch(stage, 1, i, g);
        if (a.r) fetch(stage, 2, i, along);
        if (!KEEP) weights(i, w);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const float xhat = h[j] * rho;
          dw[i][j] = fmaf(g[j], xhat, dw[i][j]);
          h[j] = rho * fmaf(-xhat, mean, g[j] * (KEEP ? kept[KEEP ? i : 0][j] : w[j])) + (a.r ? along[j] : 0.f);
        }
        NormWord<E> out;
        out.put(h);
        out.store(static_cast<E*>(a.y) + t * a.ys + (me + i * step) * U);
      }
    }
    request(stage, t + Ahead::ROWS * rows);
  }
  if (!a.partial) return;
#pragma unroll
  for (int i = 0; i < N; ++i)   // this CTA's part of dw
    if (me + i * step < all)
#pragma unroll
      for (int j = 0; j < U; j += 4)
        *reinterpret_cast<float4*>(a.partial + (int64_t)blockIdx.x * a.C + (me + i * step) * U + j) =
            make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
}

// Rows of any length, stride and alignment: a CTA a row, a value at a time, the row read again for each use.
template <typename E> __global__ void __launch_bounds__(NORM_GENERAL) norm_fwd_general_kernel(const NormArgs a) {
  chain_kernel();
  __shared__ float words[2][32];
  const int lane = threadIdx.x & 31;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* x = static_cast<const E*>(a.x) + t * a.xs;
    E* h = a.h ? static_cast<E*>(a.h) + t * a.hs : nullptr;
    float ss = 0.f;
    for (int c = threadIdx.x; c < a.C; c += NORM_GENERAL) {
      float v = to_f32(x[c]);
      if (a.r) v += to_f32(static_cast<const E*>(a.r)[t * a.rs + c]);
      const E e = from_f32<E>(v);
      if (h) h[c] = e;
      v = to_f32(e);
      ss = fmaf(v, v, ss);
    }
    const float rho = norm_inverse(over_row<false>(ss, false, words[0]), a.C, a.eps);
    const E* held = h ? h : x;
    float m = 0.f;
    for (int c = threadIdx.x; c < a.C; c += NORM_GENERAL) {
      const float z = to_f32(held[c]) * rho * a.w[c];
      m = fmaxf(m, fabsf(z));
      if (a.y) static_cast<E*>(a.y)[t * a.ys + c] = from_f32<E>(z);
    }
    if (!a.y8) continue;
    if (a.group == a.C) {
      m = fmaxf(over_row<true>(m, false, words[1]), NORM_E4M3 * NORM_LEAST);
      if (threadIdx.x == 0) a.scales[t] = m / NORM_E4M3;
      const float f = NORM_E4M3 / m;
      for (int c = threadIdx.x; c < a.C; c += NORM_GENERAL)
        a.y8[t * a.C + c] = (uint8_t)e4m3_pair(to_f32(held[c]) * rho * a.w[c] * f, 0.f);
    } else {
      const int groups = a.C / a.group;   // a warp a group; what other threads wrote of h is there since over_row
      for (int k = threadIdx.x >> 5; k < groups; k += NORM_GENERAL / 32) {
        m = 0.f;
        for (int c = k * a.group + lane; c < (k + 1) * a.group; c += 32) m = fmaxf(m, fabsf(to_f32(held[c]) * rho * a.w[c]));
        m = fmaxf(over_warp<true>(m), NORM_E4M3 * NORM_LEAST);
        if (lane == 0) a.scales[t * groups + k] = m / NORM_E4M3;
        const float f = NORM_E4M3 / m;
        for (int c = k * a.group + lane; c < (k + 1) * a.group; c += 32)
          a.y8[t * a.C + c] = (uint8_t)e4m3_pair(to_f32(held[c]) * rho * a.w[c] * f, 0.f);
      }
    }
  }
}

// (partial: each CTA adds its rows in order to its own row of sums, which begins as zeros)
template <typename E> __global__ void __launch_bounds__(NORM_GENERAL) norm_bwd_general_kernel(const NormArgs a) {
  chain_kernel();
  __shared__ float words[2][32];
  float* dw = a.partial ? a.partial + (int64_t)blockIdx.x * a.C : nullptr;
  if (dw)
    for (int c = threadIdx.x; c < a.C; c += NORM_GENERAL) dw[c] = 0.f;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* h = static_cast<const E*>(a.x) + t * a.xs;
    const E* g = static_cast<const E*>(a.dy) + t * a.hs;
    float ss = 0.f, sg = 0.f;
    for (int c = threadIdx.x; c < a.C; c += NORM_GENERAL) {
      const float v = to_f32(h[c]);
      ss = fmaf(v, v, ss);
      sg = fmaf(to_f32(g[c]) * a.w[c], v, sg);
    }
    ss = over_row<false>(ss, false, words[0]);
    const float rho = norm_inverse(ss, a.C, a.eps), mean = over_row<false>(sg, false, words[1]) * rho / (float)a.C;
    for (int c = threadIdx.x; c < a.C; c += NORM_GENERAL) {
      const float xhat = to_f32(h[c]) * rho, gv = to_f32(g[c]);
      if (dw) dw[c] = fmaf(gv, xhat, dw[c]);
      float d = rho * fmaf(-xhat, mean, gv * a.w[c]);
      if (a.r) d += to_f32(static_cast<const E*>(a.r)[t * a.rs + c]);
      static_cast<E*>(a.y)[t * a.ys + c] = from_f32<E>(d);
    }
  }
}

// dw[c] = sum over the CTAs' parts, in a fixed order: 8 runs of them side by side, then the runs in turn
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* partial, float* dw, int parts, int C) {
  chain_kernel();
  __shared__ float runs[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  float s = 0.f;
  if (c < C)
    for (int k = run; k < parts; k += 8) s += partial[(int64_t)k * C + c];
  runs[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run == 0 && c < C) {
    for (int k = 1; k < 8; ++k) s += runs[k][threadIdx.x];
    dw[c] = s;
  }
}

struct NormShape {
  bool fast;
  int vpt, threads, warp, ctas;
};

// Rows in pieces of 8 values.  Up to 64 pieces a warp takes a row.  From there to 128 a CTA does, whose rows come in whole (60,000
// BF16 rows of 1,024: 77 us, by warps 94; 100 of them 2.2 and 2.8), unless its last round is far from full (3,000 rows: 6.0 us,
// by warps 4.2) or the rows are FP32, forward (60,000: 176 us, by warps 150).  Longer ones: forward 1 piece a thread where there
// are no more rows than SMs and only latency counts (64 of 4,096: 2.5 us, 2 pieces 2.8), 2 as far as its threads go, else 4
// (20,000 rows of 12,288: 2 pieces 368 us, 4 526).
static NormShape norm_shape(const gdn_norm_problem* p, bool fast, bool back) {
  NormShape s = {fast, 0, 0, 0, 0};
  const int64_t sms = sm_count();
  const int pieces = p->C / 8;
  if (!fast || p->C > 16384) {
    s.fast = false;
    s.threads = NORM_GENERAL;
    s.ctas = (int)(p->T < sms * 4 ? p->T : sms * 4);
    return s;
  }
  // One round of CTAs, by the kernels' registers (FP32 rows of 4,096 in 1 1/3: 395 us for 309) and shared memory; backward 16-bit
  // rows 768 threads an SM (30,000 rows of 1,536 70 us, with 512 84), the shortest 512 (60,000 of 1,024 92 us, with 768 110).
  auto round_of = [&](int vpt, int threads) {
    const bool fp32 = p->dtype == GDN_FP32;
    const int resident = vpt == 4 || (back && (fp32 || threads < 96)) ? 512 : back || (fp32 && vpt == 2) ? 768 : 1024;
    return sms * (resident / threads > 0 ? resident / threads : 1);
  };
  const int64_t small = round_of(2, 64);
  const bool even = p->T <= small || (p->T + small - 1) / small * small * 20 <= p->T * 23;
  if (pieces <= 64 || (pieces <= 128 && (!even || (!back && p->dtype == GDN_FP32 && p->T > sms)))) {
    s.warp = 1;
    s.vpt = pieces <= 32 ? 1 : pieces <= 64 ? 2 : 4;
    s.threads = 128;
    const int64_t need = (p->T + 3) / 4, most = sms * (back ? 4 : 8);
    s.ctas = (int)(need < most ? need : most);
    return s;
  }
  const int two = !back && p->dtype != GDN_FP32 ? 2048 : 1024;   // pieces
  s.vpt = !back && p->T <= sms && pieces <= 1024 ? 1 : pieces <= two ? 2 : 4;
  s.threads = ((pieces + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  const int64_t most = round_of(s.vpt, s.threads);
  s.ctas = (int)(p->T < most ? p->T : most);
  return s;
}

static bool norm_check(const gdn_norm_problem* p, gdn_status* st) {
  *st = GDN_ERR_INVALID_ARG;
  if (!p || p->T < 0 || p->C < 1 || !(p->eps >= 0.f) || p->group < 0) return false;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP16 && p->dtype != GDN_FP32) return false;
  if (p->group > 0 && p->C % p->group != 0) return false;
  *st = GDN_ERR_UNSUPPORTED;
  if (p->group != 0 && p->group != 32 && p->group != 64 && p->group != 128) return false;
  if (p->T > (int64_t)INT32_MAX / 2 || p->C > 1 << 20) return false;
  *st = GDN_OK;
  return true;
}

static bool norm_stride(int64_t* s, int C) {
  if (*s == 0) *s = C;
  return *s >= C;
}

static bool on_elements(const void* p, int es) { return p && (uintptr_t)p % es == 0; }

template <typename E, bool BACK> static cudaError_t norm_run(const NormArgs& a, const NormShape& s, cudaStream_t st) {
  const dim3 grid(s.ctas), block(s.threads);
  if (!s.fast) return launch_chained(BACK ? norm_bwd_general_kernel<E> : norm_fwd_general_kernel<E>, grid, block, 0, st, a);
  if constexpr (BACK) {
    const size_t smem = s.warp && a.partial ? (size_t)(s.threads / 32) * a.C * sizeof(float) : 0;
    auto by_rows = [&](auto pieces) {
      constexpr int V = decltype(pieces)::value;
      const size_t bytes = (size_t)NormAhead<E, V>::BYTES * s.threads;
      const cudaError_t e =
          cudaFuncSetAttribute(norm_bwd_rows_kernel<E, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, NormAhead<E, V>::BYTES * 512);
      return e != cudaSuccess ? e : launch_chained(norm_bwd_rows_kernel<E, V>, grid, block, bytes, st, a);
    };
    if (!s.warp) return s.vpt == 2 ? by_rows(std::integral_constant<int, 2>()) : by_rows(std::integral_constant<int, 4>());
    if (s.vpt == 1) return launch_chained(norm_bwd_kernel<E, 1>, grid, block, smem, st, a);
    if (s.vpt == 2) return launch_chained(norm_bwd_kernel<E, 2>, grid, block, smem, st, a);
    return launch_chained(norm_bwd_kernel<E, 4>, grid, block, smem, st, a);
  } else {
#define GDN_NORM(V, W) return launch_chained(norm_fwd_kernel<E, V, W>, grid, block, 0, st, a)
    if (s.warp) {
      if (s.vpt == 1) GDN_NORM(1, true);
      if (s.vpt == 2) GDN_NORM(2, true);
      GDN_NORM(4, true);
    }
    if (s.vpt == 1) GDN_NORM(1, false);
    if constexpr (sizeof(E) == 4) {   // (16-bit rows have threads enough for 2)
      if (s.vpt == 4) GDN_NORM(4, false);
    }
    GDN_NORM(2, false);
#undef GDN_NORM
  }
}

template <bool BACK> static cudaError_t norm_by_type(int dtype, const NormArgs& a, const NormShape& s, cudaStream_t st) {
  if (dtype == GDN_BF16) return norm_run<__nv_bfloat16, BACK>(a, s, st);
  if (dtype == GDN_FP16) return norm_run<__half, BACK>(a, s, st);
  return norm_run<float, BACK>(a, s, st);
}

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_add_norm_workspace_bytes(const gdn_norm_problem* p, size_t* bytes) {
  gdn_status st;
  if (!norm_check(p, &st)) return st;
  if (!bytes) return GDN_ERR_INVALID_ARG;
  const int fast = norm_shape(p, p->C % 8 == 0, true).ctas, general = norm_shape(p, false, true).ctas;
  *bytes = (size_t)(fast > general ? fast : general) * p->C * sizeof(float);   // (alignment decides which kernel it is)
  return GDN_OK;
}

gdn_status gdn_add_norm_fwd(const gdn_norm_problem* p, const void* x, const void* r, const float* w, void* h, void* y,
                            void* y8, float* scales, struct CUstream_st* stream) {
  gdn_status st;
  if (!norm_check(p, &st)) return st;
  const int es = elem_bytes(p->dtype);
  NormArgs a = {};
  a.xs = p->x_stride, a.rs = p->r_stride, a.hs = p->h_stride, a.ys = p->y_stride;
  if (!norm_stride(&a.xs, p->C) || !norm_stride(&a.rs, p->C) || !norm_stride(&a.hs, p->C) || !norm_stride(&a.ys, p->C))
    return GDN_ERR_INVALID_ARG;
  if ((r && !h) || (!h && !y && !y8) || !y8 != !scales) return GDN_ERR_INVALID_ARG;
  if (p->T == 0) return GDN_OK;
  if (!on_elements(x, es) || (r && !on_elements(r, es)) || (h && !on_elements(h, es)) || (y && !on_elements(y, es)) || !w ||
      !on_words(w, scales))
    return GDN_ERR_INVALID_ARG;
  a.x = x, a.r = r, a.w = w, a.h = h, a.y = y, a.y8 = static_cast<uint8_t*>(y8), a.scales = scales;
  a.T = p->T, a.C = p->C, a.group = p->group ? p->group : p->C, a.eps = p->eps;
  auto rows16 = [&](const void* q, int64_t stride) { return !q || (aligned16(q) && stride * es % 16 == 0); };
  const bool fast = p->C % 8 == 0 && rows16(x, a.xs) && rows16(r, a.rs) && rows16(h, a.hs) && rows16(y, a.ys) && aligned16(w) &&
                    (uintptr_t)y8 % 8 == 0;
  prof_begin(K_NORM_FWD, stream);
  const cudaError_t e = norm_by_type<false>(p->dtype, a, norm_shape(p, fast, false), stream);
  prof_end(K_NORM_FWD, stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_add_norm_bwd(const gdn_norm_problem* p, const void* h, const float* w, const void* dy, const void* dres,
                            void* dx, float* dw, void* workspace, size_t ws_bytes, struct CUstream_st* stream) {
  gdn_status st;
  if (!norm_check(p, &st)) return st;
  const int es = elem_bytes(p->dtype);
  NormArgs a = {};
  a.xs = p->h_stride, a.rs = p->r_stride, a.hs = p->y_stride, a.ys = p->x_stride;
  if (!norm_stride(&a.xs, p->C) || !norm_stride(&a.rs, p->C) || !norm_stride(&a.hs, p->C) || !norm_stride(&a.ys, p->C))
    return GDN_ERR_INVALID_ARG;
  if (dw && !on_words(dw)) return GDN_ERR_INVALID_ARG;
  if (p->T > 0 && (!on_elements(h, es) || !on_elements(dy, es) || (dres && !on_elements(dres, es)) || !on_elements(dx, es) ||
                   !w || !on_words(w)))
    return GDN_ERR_INVALID_ARG;
  size_t need = 0;
  if (dw && p->T > 0) {
    if (!aligned16(workspace)) return GDN_ERR_INVALID_ARG;
    gdn_add_norm_workspace_bytes(p, &need);
    if (ws_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
  }
  if (p->T == 0) {
    if (dw && cudaMemsetAsync(dw, 0, (size_t)p->C * sizeof(float), stream) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
  }
  a.x = h, a.r = dres, a.dy = dy, a.w = w, a.y = dx, a.partial = dw ? static_cast<float*>(workspace) : nullptr;
  a.T = p->T, a.C = p->C, a.eps = p->eps;
  auto rows16 = [&](const void* q, int64_t stride) { return !q || (aligned16(q) && stride * es % 16 == 0); };
  const bool fast = p->C % 8 == 0 && rows16(h, a.xs) && rows16(dy, a.hs) && rows16(dres, a.rs) && rows16(dx, a.ys) && aligned16(w);
  const NormShape s = norm_shape(p, fast, true);
  prof_begin(K_NORM_BWD, stream);
  cudaError_t e = norm_by_type<true>(p->dtype, a, s, stream);
  if (e == cudaSuccess && dw)
    e = launch_chained(norm_reduce_kernel, dim3((p->C + 31) / 32), dim3(256), 0, stream, (const float*)workspace, dw, s.ctas, p->C);
  prof_end(K_NORM_BWD, stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
