// gdn_qk.cu -- the norm of q and k per head with the position rotation in the same pass (forward),
// and the host layer of both directions.
//
// Per row x of D values: r = 1 / sqrt(share x.x + eps), z = w x r, and each rotated pair of z turned by the
// token's angle.  With the token's cos and sin and the weights folded into two coefficients a value,
//   y[i] = r (x[i] (w[i] co[i]) + x[i'] (w[i'] si[i]))   (i' the partner of i),
// a row costs one sum of squares, its partners and two multiply-adds a value.
//
// Fast kernel: bandwidth-bound, every value read and written once.  A row lies in L lanes of 8 or 24 values; a group of
// L lanes takes a token and walks its heads with the token's coefficients in registers, while the next rows
// are on their way into the warp's ring in shared memory.  A warp stays with q or with k, and waits for no
// other. Few tokens: their heads are split over warps.  PLAIN: a norm and the whole row rotated, which
// needs no masks.
// The kernel for other rows (any alignment, odd D, rot not a multiple of 4 in the half layout) spreads a row over a
// warp, value by value, and takes partners from shared memory.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "gdn_launch.cuh"
#include "gdn_prof.h"
#include "gdn_qk.cuh"

namespace gdn {

template <typename E, int L, int M, int LAYOUT, bool PLAIN>
__global__ void __launch_bounds__(QK_THREADS) qk_fwd_kernel(const QkArgs a) {
  chain_kernel();
  using R = Ring<E, L, 1, M>;
  constexpr int VEC = 16 / (int)sizeof(E);   // values of one copy
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
  E* ybase = static_cast<E*>(which ? a.out[1] : a.out[0]);
  const int64_t xt = which ? a.xt[1] : a.xt[0], xh = which ? a.xh[1] : a.xh[0];
  const int64_t yt = which ? a.yt[1] : a.yt[0], yh = which ? a.yh[1] : a.yh[0];
  Place<L> at, to;   // of the work, and of the rows that are requested
  at.unit = to.unit = cta * QK_WARPS + (threadIdx.x >> 5);
  if (at.unit >= units) return;
  to.enter(a, splits, heads);
  at = to;
  int doc = 0, pos = position_of(a, at.t, &doc);   // (a unit ahead: its load is not waited for)
  Angles<L, M, LAYOUT, sizeof(E) == 2> ang;
  ang.request(a, l);
  float2 w[M][4];
#pragma unroll
  for (int m = 0; m < M; ++m)
    piece_weights(which ? a.w[1] : a.w[0], piece, m, w[m]);
  const E* px = xbase + to.t * xt + to.h * xh;
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
        }
      px += xh;
      if (--to.left == 0) {
        to.unit += warps;
        more = to.unit < units;
        if (more) {
          to.enter(a, splits, heads);
          px = xbase + to.t * xt + to.h * xh;
        }
      }
    }
    copies_commit();
    fill = R::next(fill);
  };
  clear_ring<E, L, 1, M>(slots, a.D);
#pragma unroll
  for (int i = 0; i < R::STAGES - 1; ++i) request();

  ang.setup();
  for (;;) {
    float2 wc[M][4], ws[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float2 co[4], si[4];
      ang.at(a, pos, l, m, co, si);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wc[m][j] = __fmul2_rn(w[m][j], co[j]);
        ws[m][j] = __fmul2_rn(partner_of<LAYOUT>(w[m], j), si[j]);
      }
    }
    E* y = ybase + at.t * yt + at.h * yh;
    const bool keep = at.live;
    const int rows = at.left;
    at.unit += warps;
    if (at.unit < units) {
      at.enter(a, splits, heads);
      pos = position_of(a, at.t, &doc);
    }
    for (int n = rows; n > 0; --n) {
      copies_wait<R::STAGES - 2>();
      __syncwarp();   // every lane's share of this slot is there, and the last slot has been read by all
      request();      // into the last slot
      float2 v[M][4];
#pragma unroll
      for (int m = 0; m < M; ++m) read_piece<E, 0>(read + use, piece, m, v[m]);
      use = R::next(use);
      float r = 1.f;
      if (PLAIN || a.normed) {
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4 * M; ++j)
          s = j ? __ffma2_rn(v[j / 4][j % 4], v[j / 4][j % 4], s) : __fmul2_rn(v[0][0], v[0][0]);
        r = rsqrtf(fmaf(row_sum<L>(s.x + s.y), a.share, a.eps));
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float2 p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = partner_of<LAYOUT>(v[m], j);
        if (!PLAIN) piece.only_rotated(m, p);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[m][j] = __fmul2_rn(make_float2(r, r), __ffma2_rn(p[j], ws[m][j], __fmul2_rn(v[m][j], wc[m][j])));
        if (keep && piece.has[m]) write_piece<E>(y, piece, m, v[m]);
      }
      y += yh;
    }
    if (at.unit >= units) return;
  }
}

// rows of any kind: lane i has the values i, i + 32, ... (PER of them) of each row of its warp's token
template <typename E, int PER>
__global__ void __launch_bounds__(QK_THREADS) qk_fwd_row_kernel(const QkArgs a) {
  chain_kernel();
  __shared__ float rows[QK_WARPS][PER * 32];
  float* z = rows[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const int which = blockIdx.x >= a.ctas_q, cta = blockIdx.x - (which ? a.ctas_q : 0);
  const int warps = (which ? gridDim.x - a.ctas_q : a.ctas_q) * QK_WARPS;
  const int units = which ? a.units[1] : a.units[0];
  const int splits = which ? a.splits[1] : a.splits[0], heads = which ? a.heads[1] : a.heads[0];
  const int64_t xh = which ? a.xh[1] : a.xh[0], yh = which ? a.yh[1] : a.yh[0];
  Place<32> at;
  at.unit = cta * QK_WARPS + (threadIdx.x >> 5);
  RowAngles<PER> ang;
  ang.setup(a);
  float w[PER];
  row_weights<PER>(which ? a.w[1] : a.w[0], a.D, w);
  for (; at.unit < units; at.unit += warps) {
    at.enter(a, splits, heads);
    ang.at(a, at.t);
    const E* x = static_cast<const E*>(which ? a.x[1] : a.x[0]) + at.t * (which ? a.xt[1] : a.xt[0]) + at.h * xh;
    E* y = static_cast<E*>(which ? a.out[1] : a.out[0]) + at.t * (which ? a.yt[1] : a.yt[0]) + at.h * yh;
    for (int n = at.left; n > 0; --n, x += xh, y += yh) {
      float v[PER], ss = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[i] = lane + 32 * i < a.D ? to_f32(x[lane + 32 * i]) : 0.f;
        ss = fmaf(v[i], v[i], ss);
      }
      __syncwarp();   // the last row has been read
#pragma unroll
      for (int i = 0; i < PER; ++i) z[lane + 32 * i] = v[i] *= w[i];
      const float r = a.normed ? rsqrtf(fmaf(row_sum<32>(ss), a.share, a.eps)) : 1.f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (lane + 32 * i >= a.D) break;
        if (lane + 32 * i < a.rot) v[i] = fmaf(z[ang.partner[i]], ang.s[i], v[i] * ang.c[i]);
        y[lane + 32 * i] = from_f32<E>(r * v[i]);
      }
    }
  }
}

template <typename E, int L, int M, int LAYOUT, bool PLAIN> static void launch_fwd_kernel(QkArgs& a, cudaStream_t s) {
  static const int resident = resident_ctas(qk_fwd_kernel<E, L, M, LAYOUT, PLAIN>);
  const int ctas = divide_work(a, L, resident, 1);
  launch_chained(qk_fwd_kernel<E, L, M, LAYOUT, PLAIN>, ctas, QK_THREADS, 0, s, a);
}
template <typename E, int L, int M> static void launch_fwd_rows(QkArgs& a, cudaStream_t s) {
  const bool plain = plain_rows(a);
  if (a.half_layout && a.rot % 8 != 0) launch_fwd_kernel<E, L, M, HALF_BY_4, false>(a, s);
  else if (a.half_layout && plain) launch_fwd_kernel<E, L, M, HALF, true>(a, s);
  else if (a.half_layout) launch_fwd_kernel<E, L, M, HALF, false>(a, s);
  else if (plain) launch_fwd_kernel<E, L, M, PAIRS, true>(a, s);
  else launch_fwd_kernel<E, L, M, PAIRS, false>(a, s);
}
template <typename E, int PER> static void launch_fwd_any(QkArgs& a, cudaStream_t s) {
  static const int resident = resident_ctas(qk_fwd_row_kernel<E, PER>);
  const int ctas = divide_work(a, 32, resident, 1);
  launch_chained(qk_fwd_row_kernel<E, PER>, ctas, QK_THREADS, 0, s, a);
}
// L and M by the row's length, and three_pieces
template <typename E> static void launch_fwd(QkArgs& a, bool fast, cudaStream_t s) {
  if (!fast) return a.D <= 128 ? launch_fwd_any<E, 4>(a, s) : launch_fwd_any<E, QK_MAXD / 32>(a, s);
  if constexpr (sizeof(E) == 2) {
    if (three_pieces(a) && a.D > 64 && a.D <= 96) return launch_fwd_rows<E, 4, 3>(a, s);
    if (three_pieces(a) && a.D > 128 && a.D <= 192) return launch_fwd_rows<E, 8, 3>(a, s);
  }
  if (a.D <= 64) return launch_fwd_rows<E, 8, 1>(a, s);
  if (a.D <= 128) return launch_fwd_rows<E, 16, 1>(a, s);
  launch_fwd_rows<E, 32, 1>(a, s);
}

// ---------------------------------------------------------------------------
// host layer
// ---------------------------------------------------------------------------
static gdn_status qk_check(const gdn_qk_problem* p) {
  if (!p || p->T < 0 || p->N < 0 || p->HQ < 0 || p->HK < 0 || p->D < 1) return GDN_ERR_INVALID_ARG;
  if (p->rot < 0 || p->rot > p->D || p->rot % 2 != 0) return GDN_ERR_INVALID_ARG;
  if (p->layout != GDN_ROPE_HALF && p->layout != GDN_ROPE_PAIRS) return GDN_ERR_INVALID_ARG;
  if (p->norm != GDN_NORM_NONE && p->norm != GDN_NORM_RMS && p->norm != GDN_NORM_L2) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (p->D > QK_MAXD || p->T > (int64_t)INT32_MAX / 2 || (int64_t)p->HQ + p->HK > 65536) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

static bool vectors(const void* p, int64_t token, int64_t head, int es) {
  return ((uintptr_t)p & 15) == 0 && token * es % 16 == 0 && head * es % 16 == 0;
}

// the kernels' arguments, and whether the fast ones take the rows
static gdn_status qk_args(const gdn_qk_problem* p, const void* q, const void* k, const float* wq, const float* wk,
                          const double* freq, const int32_t* pos, const int32_t* cu, const void* inq, const void* ink,
                          void* outq, void* outk, bool back, QkArgs* a, bool* fast) {
  memset(a, 0, sizeof(*a));
  const int es = elem_bytes(p->dtype);
  const void* x[2] = {q, k};
  const void* in[2] = {inq, ink};
  void* out[2] = {outq, outk};
  const int heads[2] = {p->HQ, p->HK};
  const int64_t st[2][4] = {{p->q_token, p->q_head, p->qo_token, p->qo_head},
                            {p->k_token, p->k_head, p->ko_token, p->ko_head}};
  *fast = p->D % 8 == 0 && p->D <= QK_FAST_MAXD && (p->layout == GDN_ROPE_PAIRS || p->rot % 4 == 0);
  for (int i = 0; i < 2; ++i) {
    a->heads[i] = heads[i];
    if (heads[i] == 0) continue;
    if (!x[i] || !out[i] || (back && !in[i])) return GDN_ERR_INVALID_ARG;
    if (((uintptr_t)x[i] | (uintptr_t)out[i] | (uintptr_t)in[i]) % es != 0) return GDN_ERR_INVALID_ARG;
    for (int s = 0; s < 4; ++s)
      if (st[i][s] < 0) return GDN_ERR_INVALID_ARG;
    a->xh[i] = st[i][1] ? st[i][1] : p->D;
    a->xt[i] = st[i][0] ? st[i][0] : a->xh[i] * heads[i];
    a->yh[i] = st[i][3] ? st[i][3] : p->D;
    a->yt[i] = st[i][2] ? st[i][2] : a->yh[i] * heads[i];
    if ((heads[i] > 1 && (a->xh[i] < p->D || a->yh[i] < p->D)) || (p->T > 1 && (a->xt[i] < p->D || a->yt[i] < p->D)))
      return GDN_ERR_INVALID_ARG;
    a->x[i] = x[i];
    a->in[i] = in[i];
    a->out[i] = out[i];
    *fast = *fast && vectors(x[i], a->xt[i], a->xh[i], es) &&
            (back ? vectors(out[i], a->xt[i], a->xh[i], es) && vectors(in[i], a->yt[i], a->yh[i], es)
                  : vectors(out[i], a->yt[i], a->yh[i], es));
  }
  if (p->rot > 0 && (!freq || ((uintptr_t)freq & 7) != 0)) return GDN_ERR_INVALID_ARG;
  if ((cu && p->N < 1) || !on_words(wq, wk, pos, cu)) return GDN_ERR_INVALID_ARG;
  a->w[0] = wq;
  a->w[1] = wk;
  a->freq = freq;
  a->pos = pos;
  a->cu = cu;
  a->T = p->T;
  a->N = p->N;
  a->D = p->D;
  a->rot = p->rot;
  a->half_layout = p->layout == GDN_ROPE_HALF;
  a->normed = p->norm != GDN_NORM_NONE;
  a->share = p->norm == GDN_NORM_RMS ? 1.f / (float)p->D : p->norm == GDN_NORM_L2 ? 1.f : 0.f;
  a->eps = p->eps;
  a->mscale = p->mscale;
  return GDN_OK;
}

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_qk_workspace_bytes(const gdn_qk_problem* p, size_t* bytes) {
  const gdn_status st = qk_check(p);
  if (st != GDN_OK) return st;
  if (!bytes) return GDN_ERR_INVALID_ARG;
  // two rows of partial sums a CTA, of which there are at most so many an SM (divide_work), and a warp has at least a row
  const int64_t rows = (p->T * p->HQ + QK_WARPS - 1) / QK_WARPS + (p->T * p->HK + QK_WARPS - 1) / QK_WARPS;
  const int64_t ctas = std::max<int64_t>(2, std::min<int64_t>(rows, (int64_t)sm_count() * QK_CTAS));
  *bytes = (size_t)ctas * 2 * p->D * sizeof(float);
  return GDN_OK;
}

gdn_status gdn_qk_norm_rope_fwd(const gdn_qk_problem* p, const void* q, const void* k, const float* wq,
                                const float* wk, const double* freq, const int32_t* positions,
                                const int32_t* cu_dev, void* qo, void* ko, struct CUstream_st* stream) {
  gdn_status st = qk_check(p);
  if (st != GDN_OK) return st;
  if (p->T == 0 || p->HQ + p->HK == 0) return GDN_OK;
  QkArgs a;
  bool fast;
  st = qk_args(p, q, k, wq, wk, freq, positions, cu_dev, nullptr, nullptr, qo, ko, false, &a, &fast);
  if (st != GDN_OK) return st;
  prof_begin(K_QK_FWD, stream);
  switch (p->dtype) {
    case GDN_BF16: launch_fwd<__nv_bfloat16>(a, fast, stream); break;
    case GDN_FP16: launch_fwd<__half>(a, fast, stream); break;
    default: launch_fwd<float>(a, fast, stream); break;
  }
  prof_end(K_QK_FWD, stream);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_qk_norm_rope_bwd(const gdn_qk_problem* p, const void* q, const void* k, const float* wq,
                                const float* wk, const double* freq, const int32_t* positions,
                                const int32_t* cu_dev, const void* dqo, const void* dko, void* dq, void* dk,
                                float* dwq, float* dwk, void* workspace, size_t ws_bytes,
                                struct CUstream_st* stream) {
  gdn_status st = qk_check(p);
  if (st != GDN_OK) return st;
  if ((dwq && ((uintptr_t)dwq & 3)) || (dwk && ((uintptr_t)dwk & 3))) return GDN_ERR_INVALID_ARG;
  size_t need = 0;
  gdn_qk_workspace_bytes(p, &need);
  if ((dwq || dwk) && ws_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if ((dwq || dwk) && !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
  if (p->T == 0 || p->HQ + p->HK == 0) {   // no rows: the weights' gradients are zero
    if (dwq && cudaMemsetAsync(dwq, 0, sizeof(float) * p->D, stream) != cudaSuccess) return GDN_ERR_CUDA;
    if (dwk && cudaMemsetAsync(dwk, 0, sizeof(float) * p->D, stream) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
  }
  QkArgs a;
  bool fast;
  st = qk_args(p, q, k, wq, wk, freq, positions, cu_dev, dqo, dko, dq, dk, true, &a, &fast);
  if (st != GDN_OK) return st;
  a.part = dwq || dwk ? static_cast<float*>(workspace) : nullptr;
  prof_begin(K_QK_BWD, stream);
  launch_qk_bwd(a, p->dtype, fast, dwq, dwk, stream);
  prof_end(K_QK_BWD, stream);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original,
                                double fast, double slow, double* freq, float* mscale) {
  if (rot < 0 || rot % 2 != 0 || !(base > 0.0) || !std::isfinite(base) || !freq || !mscale) return GDN_ERR_INVALID_ARG;
  if (scaling != GDN_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return GDN_ERR_INVALID_ARG;
  const double two_pi = 2.0 * std::acos(-1.0);
  double low = 0.0, high = 0.0;
  *mscale = 1.f;
  switch (scaling) {
    case GDN_ROPE_PLAIN:
    case GDN_ROPE_LINEAR: break;
    case GDN_ROPE_BASE:
      if (rot <= 2) return GDN_ERR_INVALID_ARG;
      base *= std::pow(factor, (double)rot / (rot - 2));
      break;
    case GDN_ROPE_PARTS:
      if (!(original > 0.0) || !(slow > 0.0) || !(fast >= slow) || !std::isfinite(fast) || !std::isfinite(original) ||
          base <= 1.0 || factor < 1.0)
        return GDN_ERR_INVALID_ARG;
      // the pair index whose frequency turns n times within the trained length
      low = std::max(0.0, std::floor(rot * std::log(original / (fast * two_pi)) / (2.0 * std::log(base))));
      high = std::min(rot - 1.0, std::ceil(rot * std::log(original / (slow * two_pi)) / (2.0 * std::log(base))));
      *mscale = (float)(0.1 * std::log(factor) + 1.0);
      break;
    default: return GDN_ERR_INVALID_ARG;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == GDN_ROPE_LINEAR) f /= factor;
    if (scaling == GDN_ROPE_PARTS) {
      const double ramp = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 1e-3)));
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    freq[i] = f;
  }
  return GDN_OK;
}

}  // extern "C"
