// gdn_qk_bwd.cu -- the gradients of the norm with rotation (gdn_qk.cu).
//
// With g' the output's gradient turned back by the token's angle, x^ = x r and c the norm's share:
//   dx = r (w g' - x^ c sum(w g' x^)),   dw = sum over tokens and heads of g' x^.
// One pass reads x and the gradient and writes dx: a row's two sums, x.x and (w g').x, are reduced
// together.  Work and layout are the forward's.  Each lane keeps its values' share of dwq and dwk in registers
// over all its rows; they are added over the CTA's lane groups in order, written as one partial a CTA, and a second
// kernel adds the partials in order, so results do not depend on scheduling.
#include "gdn_launch.cuh"
#include "gdn_prof.h"
#include "gdn_qk.cuh"

namespace gdn {

template <typename E, int L, int M, int LAYOUT, bool PLAIN>
__global__ void __launch_bounds__(QK_THREADS) qk_bwd_kernel(const QkArgs a) {
  chain_kernel();
  using R = Ring<E, L, 2, M>;
  constexpr int VEC = 16 / (int)sizeof(E);
  __shared__ __align__(16) E ring[QK_WARPS][R::STAGES][R::SLOT];
  E* slots = ring[threadIdx.x >> 5][0];
  const int l = threadIdx.x % L, mine = (threadIdx.x & 31) / L * R::ROW;
  Pieces<L, M, LAYOUT> piece;
  piece.setup(a, l);
  const int which = blockIdx.x >= a.ctas_q, cta = blockIdx.x - (which ? a.ctas_q : 0);
  const int warps = (which ? gridDim.x - a.ctas_q : a.ctas_q) * QK_WARPS;
  const int units = which ? a.units[1] : a.units[0];
  const int splits = which ? a.splits[1] : a.splits[0], heads = which ? a.heads[1] : a.heads[0];
  const E* xbase = static_cast<const E*>(which ? a.x[1] : a.x[0]) + l * VEC;
  const E* gbase = static_cast<const E*>(which ? a.in[1] : a.in[0]) + l * VEC;
  E* dbase = static_cast<E*>(which ? a.out[1] : a.out[0]);
  const int64_t xt = which ? a.xt[1] : a.xt[0], xh = which ? a.xh[1] : a.xh[0];
  const int64_t yt = which ? a.yt[1] : a.yt[0], yh = which ? a.yh[1] : a.yh[0];
  float2 acc[M][4];
#pragma unroll
  for (int j = 0; j < 4 * M; ++j) acc[j / 4][j % 4] = make_float2(0.f, 0.f);
  Place<L> at, to;
  at.unit = to.unit = cta * QK_WARPS + (threadIdx.x >> 5);
  if (at.unit < units) {
    to.enter(a, splits, heads);
    at = to;
    int doc = 0, pos = position_of(a, at.t, &doc);   // (a unit ahead)
    Angles<L, M, LAYOUT, sizeof(E) == 2> ang;
    ang.request(a, l);
    float2 w[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
      piece_weights(which ? a.w[1] : a.w[0], piece, m, w[m]);
    const E* px = xbase + to.t * xt + to.h * xh;
    const E* pg = gbase + to.t * yt + to.h * yh;
    const uint32_t read = (uint32_t)__cvta_generic_to_shared(slots + mine);
    int fill = 0, use = 0;   // byte offsets of slots
    bool more = true;
    const uint32_t landing = (uint32_t)__cvta_generic_to_shared(slots) + (mine + l * VEC) * (int)sizeof(E);
    auto request = [&] {
      if (more) {
#pragma unroll
        for (int i = 0; i < R::CHUNKS; ++i)
          if ((l + i * L) * VEC < a.D) {   // lanes past the row's end have none of its chunks
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
    clear_ring<E, L, 2, M>(slots, a.D);
#pragma unroll
    for (int i = 0; i < R::STAGES - 1; ++i) request();

    ang.setup();
    do {
      float2 co[M][4], si[M][4];
#pragma unroll
      for (int m = 0; m < M; ++m) ang.at(a, pos, l, m, co[m], si[m]);
      E* dx = dbase + at.t * xt + at.h * xh;
      const bool live = at.live;
      const int rows = at.left;
      at.unit += warps;
      if (at.unit < units) {
        at.enter(a, splits, heads);
        pos = position_of(a, at.t, &doc);
      }
      for (int n = rows; n > 0; --n) {
        copies_wait<R::STAGES - 2>();
        __syncwarp();
        request();
        float2 v[M][4], g[M][4], gv[M][4];
        float2 s = make_float2(0.f, 0.f), d = s;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          read_piece<E, 0>(read + use, piece, m, v[m]);
          read_piece<E, R::BYTES / 2>(read + use, piece, m, g[m]);
        }
        use = R::next(use);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          // turned back: by the opposite sine
          float2 p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 o = partner_of<LAYOUT>(g[m], j);
            p[j] = make_float2(-o.x, -o.y);
          }
          if (!PLAIN) piece.only_rotated(m, p);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g[m][j] = __ffma2_rn(p[j], si[m][j], __fmul2_rn(g[m][j], co[m][j]));
            s = m + j ? __ffma2_rn(v[m][j], v[m][j], s) : __fmul2_rn(v[m][j], v[m][j]);
            gv[m][j] = __fmul2_rn(g[m][j], v[m][j]);
            d = __ffma2_rn(gv[m][j], w[m][j], d);
          }
        }
        float r = 1.f, f = 0.f;
        if (PLAIN || a.normed) {
          r = rsqrtf(fmaf(row_sum<L>(s.x + s.y), a.share, a.eps));
          f = -row_sum<L>(d.x + d.y) * a.share * r * r * r;
        }
        const float2 rr = make_float2(r, r), ff = make_float2(f, f);
        if (live) {
#pragma unroll
          for (int j = 0; j < 4 * M; ++j) acc[j / 4][j % 4] = __ffma2_rn(gv[j / 4][j % 4], rr, acc[j / 4][j % 4]);
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = __fmul2_rn(__fmul2_rn(g[m][j], w[m][j]), rr);
            v[m][j] = PLAIN || a.normed ? __ffma2_rn(v[m][j], ff, x) : x;
          }
          if (live && piece.has[m]) write_piece<E>(dx, piece, m, v[m]);
        }
        dx += xh;
      }
    } while (at.unit < units);
  }
  if (!a.part) return;
  constexpr int GROUPS = QK_THREADS / L;
  __shared__ float sums[GROUPS][L * M * 8];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // (places below L * M * 8 in lanes without values, too)
      const int d = piece.place(m, j);
      sums[threadIdx.x / L][d] = acc[m][j].x;
      sums[threadIdx.x / L][d + 1] = acc[m][j].y;
    }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += QK_THREADS) {
    float s = 0.f;
    for (int g = 0; g < GROUPS; ++g) s += sums[g][d];
    a.part[((int64_t)blockIdx.x * 2 + which) * a.D + d] = s;
  }
}

// rows of any kind, as in the forward
template <typename E, int PER>
__global__ void __launch_bounds__(QK_THREADS) qk_bwd_row_kernel(const QkArgs a) {
  chain_kernel();
  __shared__ float rows[QK_WARPS][PER * 32];
  const int lane = threadIdx.x & 31;
  float* z = rows[threadIdx.x >> 5];
  const int which = blockIdx.x >= a.ctas_q, cta = blockIdx.x - (which ? a.ctas_q : 0);
  const int warps = (which ? gridDim.x - a.ctas_q : a.ctas_q) * QK_WARPS;
  const int units = which ? a.units[1] : a.units[0];
  const int splits = which ? a.splits[1] : a.splits[0], heads = which ? a.heads[1] : a.heads[0];
  const int64_t xh = which ? a.xh[1] : a.xh[0], yh = which ? a.yh[1] : a.yh[0];
  Place<32> at;
  at.unit = cta * QK_WARPS + (threadIdx.x >> 5);
  RowAngles<PER> ang;
  ang.setup(a);
  float w[PER], acc[PER];
  row_weights<PER>(which ? a.w[1] : a.w[0], a.D, w);
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  for (; at.unit < units; at.unit += warps) {
    at.enter(a, splits, heads);
    ang.at(a, at.t);
    const int64_t first = at.t * (which ? a.xt[1] : a.xt[0]) + at.h * xh;
    const E* x = static_cast<const E*>(which ? a.x[1] : a.x[0]) + first;
    E* dx = static_cast<E*>(which ? a.out[1] : a.out[0]) + first;
    const E* gy = static_cast<const E*>(which ? a.in[1] : a.in[0]) + at.t * (which ? a.yt[1] : a.yt[0]) + at.h * yh;
    for (int n = at.left; n > 0; --n, x += xh, dx += xh, gy += yh) {
      float v[PER], g[PER], ss = 0.f, dot = 0.f;
      __syncwarp();   // the last row has been read
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[i] = lane + 32 * i < a.D ? to_f32(x[lane + 32 * i]) : 0.f;
        z[lane + 32 * i] = g[i] = lane + 32 * i < a.D ? to_f32(gy[lane + 32 * i]) : 0.f;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        // turned back: by the opposite sine
        if (lane + 32 * i < a.rot) g[i] = fmaf(-z[ang.partner[i]], ang.s[i], g[i] * ang.c[i]);
        ss = fmaf(v[i], v[i], ss);
        dot = fmaf(g[i] * w[i], v[i], dot);
      }
      float r = 1.f, f = 0.f;
      if (a.normed) {
        r = rsqrtf(fmaf(row_sum<32>(ss), a.share, a.eps));
        f = row_sum<32>(dot) * a.share * r * r;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (lane + 32 * i >= a.D) break;
        acc[i] = fmaf(g[i], v[i] * r, acc[i]);
        dx[lane + 32 * i] = from_f32<E>(r * (g[i] * w[i] - (a.normed ? v[i] * f : 0.f)));
      }
    }
  }
  if (!a.part) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) z[lane + 32 * i] = acc[i];
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += QK_THREADS) {
    float s = 0.f;
    for (int g = 0; g < QK_WARPS; ++g) s += rows[g][d];
    a.part[((int64_t)blockIdx.x * 2 + which) * a.D + d] = s;
  }
}

// dw[d] = sum over the CTAs' partials, DW_COLS columns of dwq | dwk a CTA and DW_ROWS threads a column, so that a thread's
// own sum is a few loads deep (3,648 CTAs' partials out of DRAM: 32 columns and 32 threads 10.3 us, so 8.6); q's
// partials are in CTAs 0 .. ctas_q-1, k's in the others
constexpr int DW_COLS = 8, DW_ROWS = 128;
__global__ void __launch_bounds__(DW_COLS * DW_ROWS) qk_dw_kernel(const float* part, int ctas_q, int ctas, int D,
                                                                  float* dwq, float* dwk) {
  chain_kernel();
  __shared__ float sums[DW_ROWS][DW_COLS + 1];
  const int col = blockIdx.x * DW_COLS + threadIdx.x, ty = threadIdx.y;
  float s = 0.f;
  if (col < 2 * D) {
    const int end = col < D ? ctas_q : ctas;
#pragma unroll 8
    for (int b = (col < D ? 0 : ctas_q) + ty; b < end; b += DW_ROWS) s += part[(int64_t)b * 2 * D + col];
  }
  sums[ty][threadIdx.x] = s;
#pragma unroll
  for (int half = DW_ROWS / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (ty < half) sums[ty][threadIdx.x] += sums[ty + half][threadIdx.x];
  }
  if (ty == 0 && col < 2 * D) {
    float* dw = col < D ? dwq : dwk;
    if (dw) dw[col < D ? col : col - D] = sums[0][threadIdx.x];
  }
}

template <typename E, int L, int M, int LAYOUT, bool PLAIN> static int launch_bwd_kernel(QkArgs& a, cudaStream_t s) {
  static const int resident = resident_ctas(qk_bwd_kernel<E, L, M, LAYOUT, PLAIN>);
  const int ctas = divide_work(a, L, resident, 2);
  launch_chained(qk_bwd_kernel<E, L, M, LAYOUT, PLAIN>, ctas, QK_THREADS, 0, s, a);
  return ctas;
}
template <typename E, int L, int M> static int launch_bwd_rows(QkArgs& a, cudaStream_t s) {
  const bool plain = plain_rows(a);
  if (a.half_layout && a.rot % 8 != 0) return launch_bwd_kernel<E, L, M, HALF_BY_4, false>(a, s);
  if (a.half_layout && plain) return launch_bwd_kernel<E, L, M, HALF, true>(a, s);
  if (a.half_layout) return launch_bwd_kernel<E, L, M, HALF, false>(a, s);
  if (plain) return launch_bwd_kernel<E, L, M, PAIRS, true>(a, s);
  return launch_bwd_kernel<E, L, M, PAIRS, false>(a, s);
}
template <typename E, int PER> static int launch_bwd_any(QkArgs& a, cudaStream_t s) {
  static const int resident = resident_ctas(qk_bwd_row_kernel<E, PER>);
  const int ctas = divide_work(a, 32, resident, 2);
  launch_chained(qk_bwd_row_kernel<E, PER>, ctas, QK_THREADS, 0, s, a);
  return ctas;
}
// returns the CTAs, each of which has left partial sums (L and M by the row's length, and three_pieces)
template <typename E> static int launch_bwd(QkArgs& a, bool fast, cudaStream_t s) {
  if (!fast) return a.D <= 128 ? launch_bwd_any<E, 4>(a, s) : launch_bwd_any<E, QK_MAXD / 32>(a, s);
  if constexpr (sizeof(E) == 2) {
    if (three_pieces(a) && a.D > 64 && a.D <= 96) return launch_bwd_rows<E, 4, 3>(a, s);
    if (three_pieces(a) && a.D > 128 && a.D <= 192) return launch_bwd_rows<E, 8, 3>(a, s);
  }
  if (a.D <= 64) return launch_bwd_rows<E, 8, 1>(a, s);
  if (a.D <= 128) return launch_bwd_rows<E, 16, 1>(a, s);
  return launch_bwd_rows<E, 32, 1>(a, s);
}

void launch_qk_bwd(QkArgs& a, int dtype, bool fast, float* dwq, float* dwk, cudaStream_t s) {
  const int ctas = dtype == GDN_BF16 ? launch_bwd<__nv_bfloat16>(a, fast, s)
                   : dtype == GDN_FP16 ? launch_bwd<__half>(a, fast, s)
                                       : launch_bwd<float>(a, fast, s);
  if (a.part)
    launch_chained(qk_dw_kernel, (2 * a.D + DW_COLS - 1) / DW_COLS, dim3(DW_COLS, DW_ROWS), 0, s, a.part, a.ctas_q, ctas, a.D, dwq, dwk);
}

}  // namespace gdn
