// gdn_qk_bwd.cu -- the gradients of the norm with rotation (gdn_qk.cu).
//
// With g' the output's gradient turned back by the token's angle, x^ = x r and c the norm's share:
//   dx = r (w g' - x^ c sum(w g' x^)),   dw = sum over tokens and heads of g' x^.
// One pass reads x and the gradient and writes dx: a row's two sums, x.x and (w g').x, are reduced
// together.  Work and layout are the forward's.  Each lane keeps its values' share of dwq and dwk in registers
// over all its rows; they are added over the CTA's lane groups in order, written as one partial a CTA, and a second
// kernel adds the partials in order, so results do not depend on scheduling.
#include "gdn_prof.h"
#include "gdn_qk.cuh"

namespace gdn {

template <typename E, int L, bool HALF, bool PLAIN>
__global__ void __launch_bounds__(QK_THREADS) qk_bwd_kernel(const QkArgs a) {
  using R = Ring<E, L, 2>;
  constexpr int VEC = 16 / (int)sizeof(E);
  __shared__ __align__(16) E ring[QK_WARPS][R::STAGES][R::SLOT];
  E* slots = ring[threadIdx.x >> 5][0];
  const int l = threadIdx.x % L, mine = (threadIdx.x & 31) / L * R::ROW;
  int off0, off1;
  block_offsets<HALF>(a, l, &off0, &off1);
  const int away = off1 - off0, rotated = HALF ? (l < a.rot / 8 ? 8 : 0) : a.rot - 8 * l;
  const bool has = PLAIN || l < a.D / 8;
  const int which = blockIdx.x >= a.ctas_q, cta = blockIdx.x - (which ? a.ctas_q : 0);
  const int warps = (which ? gridDim.x - a.ctas_q : a.ctas_q) * QK_WARPS;
  const int units = which ? a.units[1] : a.units[0];
  const int splits = which ? a.splits[1] : a.splits[0], heads = which ? a.heads[1] : a.heads[0];
  const E* xbase = static_cast<const E*>(which ? a.x[1] : a.x[0]) + l * VEC;
  const E* gbase = static_cast<const E*>(which ? a.in[1] : a.in[0]) + l * VEC;
  E* dbase = static_cast<E*>(which ? a.out[1] : a.out[0]) + off0;
  const int64_t xt = which ? a.xt[1] : a.xt[0], xh = which ? a.xh[1] : a.xh[0];
  const int64_t yt = which ? a.yt[1] : a.yt[0], yh = which ? a.yh[1] : a.yh[0];
  float2 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float2(0.f, 0.f);
  Place<L> at, to;
  at.unit = to.unit = cta * QK_WARPS + (threadIdx.x >> 5);
  if (at.unit < units) {
    to.enter(a, splits, heads);
    const E* px = xbase + to.t * xt + to.h * xh;
    const E* pg = gbase + to.t * yt + to.h * yh;
    const uint32_t read = (uint32_t)__cvta_generic_to_shared(slots + mine + off0);
    int fill = 0, use = 0;   // byte offsets of slots
    bool more = true;
    const uint32_t landing = (uint32_t)__cvta_generic_to_shared(slots) + (mine + l * VEC) * (int)sizeof(E);
    auto request = [&] {
      if (more) {
#pragma unroll
        for (int i = 0; i < R::CHUNKS; ++i)
          if (PLAIN || (l + i * L) * VEC < a.D) {   // lanes past the row's end have none of its chunks
            copy16(landing + fill + i * L * 16, px + i * L * VEC);
            copy16(landing + R::BYTES / 2 + fill + i * L * 16, pg + i * L * VEC);
          }
        px += xh;
        pg += yh;
        if (--to.left == 0) {
          to.unit += warps;
          more = to.unit < units;
          if (more) {
            to.enter(a, splits, heads);
            px = xbase + to.t * xt + to.h * xh;
            pg = gbase + to.t * yt + to.h * yh;
          }
        }
      }
      copies_commit();
      fill = R::next(fill);
    };
#pragma unroll
    for (int i = 0; i < R::STAGES - 1; ++i) request();

    Angles<HALF, sizeof(E) == 2> ang;
    ang.setup(a, l);
    float2 w[4];
    lane_weights(which ? a.w[1] : a.w[0], off0, off1, has, w);
    do {
      at.enter(a, splits, heads);
      float2 co[4], si[4];
      ang.at(a, at.t, l, co, si);
      E* dx = dbase + at.t * xt + at.h * xh;
      const bool keep = at.live && has;
      for (int n = at.left; n > 0; --n) {
        copies_wait<R::STAGES - 2>();
        __syncwarp();
        request();
        float2 v[4], g[4], p[4];
        const uint32_t s0 = read + use;
        read_row<E, HALF>(s0, away, v);
        read_row<E, HALF>(s0 + R::BYTES / 2, away, g);
        use = R::next(use);
        if (!PLAIN && !has) {
          only_rotated(v, 0);
          only_rotated(g, 0);
        }
        // turned back: by the opposite sine
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 o = partner_of<HALF>(g, j);
          p[j] = make_float2(-o.x, -o.y);
        }
        if (!PLAIN) only_rotated(p, rotated);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = __ffma2_rn(p[j], si[j], __fmul2_rn(g[j], co[j]));
        float2 s = __fmul2_rn(v[0], v[0]), d = make_float2(0.f, 0.f), gv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j) s = __ffma2_rn(v[j], v[j], s);
          gv[j] = __fmul2_rn(g[j], v[j]);
          d = __ffma2_rn(gv[j], w[j], d);
        }
        float r = 1.f, f = 0.f;
        if (PLAIN || a.normed) {
          r = rsqrtf(fmaf(row_sum<L>(s.x + s.y), a.share, a.eps));
          f = -row_sum<L>(d.x + d.y) * a.share * r * r * r;
        }
        const float2 rr = make_float2(r, r), ff = make_float2(f, f);
        if (at.live) {
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = __ffma2_rn(gv[j], rr, acc[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = __fmul2_rn(__fmul2_rn(g[j], w[j]), rr);
          v[j] = PLAIN || a.normed ? __ffma2_rn(v[j], ff, x) : x;
        }
        if (keep) write_row<E, HALF>(dx, away, v);
        dx += xh;
      }
      at.unit += warps;
    } while (at.unit < units);
  }
  if (!a.part) return;
  constexpr int GROUPS = QK_THREADS / L;
  __shared__ float sums[GROUPS][L * 8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = (j < 2 ? off0 : off1) + (j & 1) * 2;   // (below L * 8 in lanes without values, too)
    sums[threadIdx.x / L][d] = acc[j].x;
    sums[threadIdx.x / L][d + 1] = acc[j].y;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += QK_THREADS) {
    float s = 0.f;
    for (int g = 0; g < GROUPS; ++g) s += sums[g][d];
    a.part[((int64_t)blockIdx.x * 2 + which) * a.D + d] = s;
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
        angle_cos_sin<false>(step[f], p, a.mscale, &c, &s);
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

// dw[d] = sum over the CTAs' partials, 32 columns of dwq | dwk a CTA, 32 threads a column; q's partials are in
// CTAs 0 .. end_q-1, k's in begin_k .. ctas-1
__global__ void __launch_bounds__(1024) qk_dw_kernel(const float* part, int end_q, int begin_k, int ctas, int D,
                                                     float* dwq, float* dwk) {
  __shared__ float sums[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (col < 2 * D) {
    const int end = col < D ? end_q : ctas;
#pragma unroll 8
    for (int b = (col < D ? 0 : begin_k) + threadIdx.y; b < end; b += 32) s += part[(int64_t)b * 2 * D + col];
  }
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

template <typename E, int L, bool HALF, bool PLAIN> static int launch_bwd_kernel(QkArgs& a, cudaStream_t s) {
  static const int resident = resident_ctas(qk_bwd_kernel<E, L, HALF, PLAIN>);
  const int ctas = divide_work(a, L, resident);
  qk_bwd_kernel<E, L, HALF, PLAIN><<<ctas, QK_THREADS, 0, s>>>(a);
  return ctas;
}
template <typename E, int L> static int launch_bwd_rows(QkArgs& a, cudaStream_t s) {
  const bool plain = plain_rows(a, L);
  if (a.half_layout && plain) return launch_bwd_kernel<E, L, true, true>(a, s);
  if (a.half_layout) return launch_bwd_kernel<E, L, true, false>(a, s);
  if (plain) return launch_bwd_kernel<E, L, false, true>(a, s);
  return launch_bwd_kernel<E, L, false, false>(a, s);
}
// returns the CTAs, each of which has left partial sums
template <typename E> static int launch_bwd(QkArgs& a, bool fast, int row_ctas, cudaStream_t s) {
  if (fast && a.D <= 64) return launch_bwd_rows<E, 8>(a, s);
  if (fast && a.D <= 128) return launch_bwd_rows<E, 16>(a, s);
  if (fast) return launch_bwd_rows<E, 32>(a, s);
  qk_bwd_row_kernel<E><<<row_ctas, QK_ROW_WARPS * 32, 0, s>>>(a);
  return row_ctas;
}

void launch_qk_bwd(QkArgs& a, int dtype, bool fast, int row_ctas, float* dwq, float* dwk, cudaStream_t s) {
  const int ctas = dtype == GDN_BF16 ? launch_bwd<__nv_bfloat16>(a, fast, row_ctas, s)
                   : dtype == GDN_FP16 ? launch_bwd<__half>(a, fast, row_ctas, s)
                                       : launch_bwd<float>(a, fast, row_ctas, s);
  if (a.part)
    qk_dw_kernel<<<(2 * a.D + 31) / 32, dim3(32, 32), 0, s>>>(a.part, fast ? a.ctas_q : ctas, fast ? a.ctas_q : 0,
                                                              ctas, a.D, dwq, dwk);
}

}  // namespace gdn
