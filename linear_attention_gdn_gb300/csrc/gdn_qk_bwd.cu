// gdn_qk_bwd.cu -- the gradients of the norm with rotation (gdn_qk.cu).
//
// With g' the output's gradient turned back by the token's angle, x^ = x r and c the norm's share:
//   dx = r (w g' - x^ c sum(w g' x^)),   dw = sum over tokens and heads of g' x^.
// One pass reads x and the gradient and writes dx: a row's two sums, x.x and (w g').x, are reduced
// together.  Work and layout are the forward's.  Each thread keeps its channels' share of dwq and dwk in registers
// over all its rows; they are added over the CTA's groups in order, written as one partial a CTA, and a second
// kernel adds the partials in order, so results do not depend on scheduling.
#include "gdn_prof.h"
#include "gdn_qk.cuh"

namespace gdn {

template <typename E, int L, bool HALF>
__global__ void __launch_bounds__(QK_THREADS, QK_BWD_CTAS) qk_bwd_kernel(const QkArgs a) {
  extern __shared__ __align__(16) uint8_t qk_smem[];
  const int row_len = angle_row(a.rot), buf = a.tile * row_len;
  uint64_t* step = reinterpret_cast<uint64_t*>(qk_smem);
  float* angles = reinterpret_cast<float*>(step + row_len);
  for (int i = threadIdx.x; i < a.rot / 2; i += QK_THREADS) step[i] = turn_step(a.freq[i]);
  __syncthreads();
  constexpr int GROUPS = QK_THREADS / L;
  const int group = threadIdx.x / L, d0 = (threadIdx.x % L) * 8;
  const int per_token = a.items[0] + a.items[1], n_items = a.tile * per_token;
  HalfPartner<L> hp;
  if (HALF) hp.setup(a.rot);
  float acc[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
  int doc = 0, flip = 0;
  for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x, flip ^= 1) {
    float* cosv = angles + flip * 2 * buf;
    float* sinv = cosv + buf;
    fill_angles(a, step, tile, row_len, cosv, sinv, &doc);
    __syncthreads();
    for (int base = 0; base < n_items; base += GROUPS) {
      const int item = base + group, j = item / per_token, e = item - j * per_token;
      const int64_t t = tile * a.tile + j;
      const int which = e >= a.items[0];
      const int h0 = (e - (which ? a.items[0] : 0)) * a.run;
      const int heads = item < n_items && t < a.T && d0 < a.D ? min(a.run, a.heads[which] - h0) : 0;
      const int64_t xh = a.xh[which], yh = a.yh[which];
      const E* x = static_cast<const E*>(a.x[which]) + t * a.xt[which] + h0 * xh + d0;
      E* dx = static_cast<E*>(a.out[which]) + t * a.xt[which] + h0 * xh + d0;
      const E* gy = static_cast<const E*>(a.in[which]) + t * a.yt[which] + h0 * yh + d0;
      float co[8], si[8], w[8], dw[8];
      const int jj = item < n_items ? j : 0;
      thread_angles<L, HALF>(a, cosv + jj * row_len, sinv + jj * row_len, row_len, co, si);
      load_weights(a.w[which], d0, a.D, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[i] = 0.f;
      for (int u0 = 0; u0 < a.run; u0 += QK_BATCH / 2) {
        Raw8<E> rx[QK_BATCH / 2], rg[QK_BATCH / 2];
#pragma unroll
        for (int u = 0; u < QK_BATCH / 2; ++u) {
          if (u0 + u < heads) {
            rx[u].load(x + (u0 + u) * xh);
            rg[u].load(gy + (u0 + u) * yh);
          } else {
            rx[u].zero();
            rg[u].zero();
          }
        }
#pragma unroll
        for (int u = 0; u < QK_BATCH / 2; ++u) {
          if (u0 + u >= a.run) break;
          float v[8], g[8], p[8];
          rx[u].get(v);
          rg[u].get(g);
          partner<L, HALF>(hp, a, rg[u], p);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            g[i] = fmaf(p[i], -si[i], g[i] * co[i]);
            ss = fmaf(v[i], v[i], ss);
            dot = fmaf(w[i] * g[i], v[i], dot);
          }
          float r = 1.f, f = 0.f;
          if (a.normed) {
            r = rsqrtf(fmaf(row_sum<L>(ss), a.share, a.eps));
            f = row_sum<L>(dot) * a.share * r * r;
          }
          if (u0 + u < heads) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dw[i] = fmaf(g[i], v[i] * r, dw[i]);
              v[i] = r * (w[i] * g[i] - (a.normed ? v[i] * f : 0.f));
            }
            rx[u].put(v);
            rx[u].store(dx + (u0 + u) * xh);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[0][i] += which ? 0.f : dw[i];
        acc[1][i] += which ? dw[i] : 0.f;
      }
    }
  }
  if (!a.part) return;
  __shared__ float sums[GROUPS][L * 8];
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[group][d0 + i] = which ? acc[1][i] : acc[0][i];
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += QK_THREADS) {
      float s = 0.f;
      for (int g = 0; g < GROUPS; ++g) s += sums[g][d];
      a.part[((int64_t)blockIdx.x * 2 + which) * a.D + d] = s;
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(QK_ROW_WARPS * 32) qk_bwd_row_kernel(const QkArgs a) {
  __shared__ float rows[QK_ROW_WARPS][QK_MAXD];
  __shared__ float sums[QK_ROW_WARPS][QK_MAXD];
  constexpr int PER = QK_MAXD / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* gin = rows[warp];
  const int total = a.heads[0] + a.heads[1], half = a.rot / 2;
  __shared__ uint64_t step[QK_MAXD / 2];
  for (int i = threadIdx.x; i < half; i += QK_ROW_WARPS * 32) step[i] = turn_step(a.freq[i]);
  __syncthreads();
  float acc[2][PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[0][i] = acc[1][i] = 0.f;
  int doc = 0;
  const int64_t warps = (int64_t)gridDim.x * QK_ROW_WARPS;
  for (int64_t row = (int64_t)blockIdx.x * QK_ROW_WARPS + warp; row < a.T * total; row += warps) {
    const int64_t t = row / total;
    const int e = (int)(row - t * total), which = e >= a.heads[0], h = e - (which ? a.heads[0] : 0);
    const E* x = static_cast<const E*>(a.x[which]) + t * a.xt[which] + h * a.xh[which];
    E* dx = static_cast<E*>(a.out[which]) + t * a.xt[which] + h * a.xh[which];
    const E* gy = static_cast<const E*>(a.in[which]) + t * a.yt[which] + h * a.yh[which];
    for (int d = lane; d < a.D; d += 32) gin[d] = to_f32(gy[d]);
    const int p = position_of(a, t, &doc);
    __syncwarp();
    float v[PER], g[PER], ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int d = lane + 32 * i;
      v[i] = g[i] = 0.f;
      if (d >= a.D) continue;
      v[i] = to_f32(x[d]);
      g[i] = gin[d];
      if (d < a.rot) {
        const int f = a.half_layout ? (d < half ? d : d - half) : d >> 1;
        const int other = a.half_layout ? (d < half ? d + half : d - half) : d ^ 1;
        float c, s;
        angle_cos_sin(step[f], p, a.mscale, &c, &s);
        g[i] = g[i] * c + (d < other ? gin[other] : -gin[other]) * s;
      }
      ss = fmaf(v[i], v[i], ss);
      dot = fmaf(g[i] * (a.w[which] ? a.w[which][d] : 1.f), v[i], dot);
    }
    float r = 1.f, f = 0.f;
    if (a.normed) {
      r = rsqrtf(fmaf(row_sum<32>(ss), a.share, a.eps));
      f = row_sum<32>(dot) * a.share * r * r;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int d = lane + 32 * i;
      if (d >= a.D) continue;
      if (which) acc[1][i] = fmaf(g[i], v[i] * r, acc[1][i]);
      else acc[0][i] = fmaf(g[i], v[i] * r, acc[0][i]);
      const float wg = g[i] * (a.w[which] ? a.w[which][d] : 1.f);
      dx[d] = from_f32<E>(r * (wg - (a.normed ? v[i] * f : 0.f)));
    }
    __syncwarp();
  }
  if (!a.part) return;
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) sums[warp][lane + 32 * i] = which ? acc[1][i] : acc[0][i];
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += QK_ROW_WARPS * 32) {
      float s = 0.f;
      for (int g = 0; g < QK_ROW_WARPS; ++g) s += sums[g][d];
      a.part[((int64_t)blockIdx.x * 2 + which) * a.D + d] = s;
    }
  }
}

// dw[d] = sum over the CTAs' partials: 32 columns of dwq | dwk a CTA, 32 threads a column
__global__ void __launch_bounds__(1024) qk_dw_kernel(const float* part, int ctas, int D, float* dwq, float* dwk) {
  __shared__ float sums[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (col < 2 * D)
    for (int b = threadIdx.y; b < ctas; b += 32) s += part[(int64_t)b * 2 * D + col];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < 2 * D) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][threadIdx.x];
    float* dw = col < D ? dwq : dwk;
    if (dw) dw[col < D ? col : col - D] = v;
  }
}

template <typename E, int L>
static void launch_bwd_rows(const QkArgs& a, int ctas, cudaStream_t s) {
  const size_t smem = angle_smem(a.rot, a.tile);
  if (a.half_layout) qk_bwd_kernel<E, L, true><<<ctas, QK_THREADS, smem, s>>>(a);
  else qk_bwd_kernel<E, L, false><<<ctas, QK_THREADS, smem, s>>>(a);
}
template <typename E>
static void launch_bwd(const QkArgs& a, bool fast, int ctas, cudaStream_t s) {
  if (!fast) qk_bwd_row_kernel<E><<<ctas, QK_ROW_WARPS * 32, 0, s>>>(a);
  else if (a.D <= 64) launch_bwd_rows<E, 8>(a, ctas, s);
  else if (a.D <= 128) launch_bwd_rows<E, 16>(a, ctas, s);
  else launch_bwd_rows<E, 32>(a, ctas, s);
}

void launch_qk_bwd(const QkArgs& a, int dtype, bool fast, int ctas, float* dwq, float* dwk, cudaStream_t s) {
  switch (dtype) {
    case GDN_BF16: launch_bwd<__nv_bfloat16>(a, fast, ctas, s); break;
    case GDN_FP16: launch_bwd<__half>(a, fast, ctas, s); break;
    default: launch_bwd<float>(a, fast, ctas, s); break;
  }
  if (a.part) qk_dw_kernel<<<(2 * a.D + 31) / 32, dim3(32, 32), 0, s>>>(a.part, ctas, a.D, dwq, dwk);
}

}  // namespace gdn
