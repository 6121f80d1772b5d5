// gdn_la_step.cu -- linear attention with a fixed decay per head on a pool of states, for generation.
//
// Per token of a sequence and value head, with S the 128 x 128 FP32 state (rows: key channels) and a = exp(decay):
//   S = a S + k v^T,   o = scale S^T q = scale (a S_before^T q + (k.q) v)
// The second form takes the sums over the rows off the way from state to state.
//
// A warp owns COLS columns of one head's state: lane (r, c) = (lane / COLL, lane % COLL) holds the columns 4c .. 4c+3 of the
// rows 8r .. 8r+7 (and 64 more on, with 8 row lanes).  A load of the warp covers 32 or 64 contiguous bytes of a row.  The
// state is read once and stays in registers over all tokens of the sequence.  One token a sequence is bound by the states'
// bytes, longer ones by FP32 arithmetic (3 operations a state value a token, in pairs of rows).
// 96 sequences of 1 to 4 tokens, 32 heads, FP16, every state kept: 105 us, 98% of a plain copy's rate; one token of one
// sequence, 48 heads: 2.9 us among others, which is the launch and two dependent loads.
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_prof.h"
#include "gdn_sequences.cuh"

namespace gdn {

struct LaStepArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* decay;
  const int* cu;
  const int* slot_in;
  const int* slot_out;
  float* states;
  void* o;
  int* err;
  int64_t T, qs, ks, vs;
  int N, HV, G, slots;
  float scale;
};

template <int ROWL> struct LaStepLayout {
  static constexpr int COLL = 32 / ROWL, COLS = 4 * COLL, PARTS = D / COLS, ROWS = D / ROWL, GROUPS = ROWS / 8;
  static constexpr int PAIRS = ROWS / 2;
  // the first row, within a lane's, of the pair p
  static __device__ __forceinline__ int row(int p) { return p % 4 * 2 + p / 4 * 64; }
};

// AHEAD: the next token's rows are requested a token ahead
template <typename E, int ROWL, bool AHEAD>
__global__ void __launch_bounds__(32) la_step_kernel(const LaStepArgs a) {
  chain_kernel();
  using L = LaStepLayout<ROWL>;
  const int lane = threadIdx.x & 31, r = lane / L::COLL, c = lane % L::COLL;
  const int part = blockIdx.x % L::PARTS, h = blockIdx.x / L::PARTS % a.HV, n = blockIdx.x / L::PARTS / a.HV;
  int t0, t1;
  if (!sequence_bounds(a.cu, n, a.T, &t0, &t1)) {
    if (lane == 0) *a.err = ST_DEVICE;
    return;
  }
  if (t0 == t1) return;
  const int from = a.slot_in ? a.slot_in[n] : n;
  if (from < -1 || from >= a.slots) {
    if (lane == 0) *a.err = ST_DEVICE;
    return;
  }
  const int64_t slot_elems = (int64_t)a.HV * STATE_F32;
  const int64_t at = (int64_t)h * STATE_F32 + r * 8 * D + part * L::COLS + c * 4;
  float2 S[L::PAIRS][4];   // [pair of rows][column]
  if (from >= 0) {
    const float* p = a.states + from * slot_elems + at;
#pragma unroll
    for (int j = 0; j < L::PAIRS; ++j) {
      const float* row = p + L::row(j) * D;
      const float4 x = *reinterpret_cast<const float4*>(row), y = *reinterpret_cast<const float4*>(row + D);
      S[j][0] = make_float2(x.x, y.x);
      S[j][1] = make_float2(x.y, y.y);
      S[j][2] = make_float2(x.z, y.z);
      S[j][3] = make_float2(x.w, y.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4 * L::PAIRS; ++j) S[j >> 2][j & 3] = make_float2(0.f, 0.f);
  }
  const int hq = h / a.G;
  // after the sums a lane has the one of this column (lanes that differ in their lower row bits have copies)
  const bool b4 = lane & 16, b3 = lane & 8;
  const int own = part * L::COLS + c * 4 + (b4 ? 2 : 0) + (b3 ? 1 : 0);
  const bool writer = (lane & 7) < L::COLL;
  Raw8<E> rk[L::GROUPS], rq[L::GROUPS];
  RawV<E, 4> rv;
  int to;
  auto request = [&](int64_t t) {
    const E* kp = static_cast<const E*>(a.k) + t * a.ks + hq * D + r * 8;
    const E* qp = static_cast<const E*>(a.q) + t * a.qs + hq * D + r * 8;
#pragma unroll
    for (int m = 0; m < L::GROUPS; ++m) {
      rk[m].load(kp + 64 * m);
      rq[m].load(qp + 64 * m);
    }
    rv.load(static_cast<const E*>(a.v) + t * a.vs + h * D + part * L::COLS + c * 4);
    to = a.slot_out ? a.slot_out[t] : t == t1 - 1 ? from : -1;
  };
  request(t0);
  const float decay = expf(a.decay[h]);
  const float2 d2 = make_float2(decay, decay);
  E* op = static_cast<E*>(a.o) + ((int64_t)t0 * a.HV + h) * D + own;
  for (int t = t0; t < t1; ++t, op += (int64_t)a.HV * D) {
    if (!AHEAD && t > t0) request(t);
    float2 k[L::PAIRS], s[4];
    float2 kq = make_float2(0.f, 0.f);
#pragma unroll
    for (int m = 0; m < L::GROUPS; ++m) {
      float kf[8], qf[8];
      rk[m].get(kf);
      rq[m].get(qf);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = 4 * m + j;
        k[p] = make_float2(kf[2 * j], kf[2 * j + 1]);
        const float2 q = make_float2(qf[2 * j], qf[2 * j + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = p ? __ffma2_rn(S[p][i], q, s[i]) : __fmul2_rn(S[p][i], q);
        kq = __ffma2_rn(k[p], q, kq);
      }
    }
    float v[4];
    rv.get(v);
    const int dest = to;
    if (AHEAD && t + 1 < t1) request(t + 1);
#pragma unroll
    for (int j = 0; j < 4 * L::PAIRS; ++j) {
      const float2 vv = make_float2(v[j & 3], v[j & 3]);
      S[j >> 2][j & 3] = __ffma2_rn(k[j >> 2], vv, __fmul2_rn(S[j >> 2][j & 3], d2));
    }
    // sums over the row lanes; the four columns are spread over them on the way
    float x = kq.x + kq.y, w[2], y;
#pragma unroll
    for (int d = L::COLL; d <= 16; d <<= 1) x += __shfl_xor_sync(~0u, x, d);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float lo = s[i].x + s[i].y, hi = s[2 + i].x + s[2 + i].y;
      w[i] = (b4 ? hi : lo) + __shfl_xor_sync(~0u, b4 ? lo : hi, 16);
    }
    y = (b3 ? w[1] : w[0]) + __shfl_xor_sync(~0u, b3 ? w[0] : w[1], 8);
#pragma unroll
    for (int d = L::COLL; d < 8; d <<= 1) y += __shfl_xor_sync(~0u, y, d);
    const float mine = b4 ? (b3 ? v[3] : v[2]) : (b3 ? v[1] : v[0]);
    if (writer) *op = from_f32<E>(a.scale * fmaf(x, mine, decay * y));
    if (dest >= a.slots || dest < -1) {
      if (lane == 0) *a.err = ST_DEVICE;
    } else if (dest >= 0) {
      float* p = a.states + dest * slot_elems + at;
#pragma unroll
      for (int j = 0; j < L::PAIRS; ++j) {
        float* row = p + L::row(j) * D;
        *reinterpret_cast<float4*>(row) = make_float4(S[j][0].x, S[j][1].x, S[j][2].x, S[j][3].x);
        *reinterpret_cast<float4*>(row + D) = make_float4(S[j][0].y, S[j][1].y, S[j][2].y, S[j][3].y);
      }
    }
  }
}

template <typename E> static cudaError_t launch_la_step(const LaStepArgs& a, int64_t heads, cudaStream_t s) {
  // few heads: 16 row lanes, 8 columns a warp (one token of 48 heads 2.86 us, by 8 row lanes and 16 columns 3.19; of 144 5.85
  // and 4.05)
  if (heads <= sm_count() / 2)
    return launch_chained(la_step_kernel<E, 16, true>, dim3((unsigned)heads * LaStepLayout<16>::PARTS), dim3(32), 0, s, a);
  const dim3 grid((unsigned)heads * LaStepLayout<8>::PARTS);
  if (a.T <= a.N) return launch_chained(la_step_kernel<E, 8, false>, grid, dim3(32), 0, s, a);
  return launch_chained(la_step_kernel<E, 8, true>, grid, dim3(32), 0, s, a);
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_la_step(const gdn_step_problem* p, const void* q, const void* k, const void* v,
                                  const float* decay, const int32_t* cu, const int32_t* slot_in, const int32_t* slot_out,
                                  float* states, void* o, int32_t* err, struct CUstream_st* stream) {
  if (!p || p->T < 0 || p->N < 0 || p->H < 1 || p->HV < 1 || p->slots < 0) return GDN_ERR_INVALID_ARG;
  if (p->dk != D || p->dv != D || p->HV % p->H != 0 || p->T > (int64_t)INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
  if (p->l2norm) return GDN_ERR_UNSUPPORTED;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (!cu && p->T != p->N) return GDN_ERR_INVALID_ARG;
  if (!slot_in && p->slots < p->N) return GDN_ERR_INVALID_ARG;
  LaStepArgs a;
  a.qs = p->q_stride;
  a.ks = p->k_stride;
  a.vs = p->v_stride;
  const int es = elem_bytes(p->dtype);
  if (!step_stride(&a.qs, p->H, es) || !step_stride(&a.ks, p->H, es) || !step_stride(&a.vs, p->HV, es))
    return GDN_ERR_INVALID_ARG;
  if (!err) return GDN_ERR_INVALID_ARG;
  if (p->T == 0 || p->N == 0) return GDN_OK;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !decay || !aligned16(o) || (p->slots > 0 && !aligned16(states)) ||
      !on_words(decay, cu, slot_in, slot_out, err))
    return GDN_ERR_INVALID_ARG;
  const int64_t heads = (int64_t)p->N * p->HV;
  if (heads * LaStepLayout<16>::PARTS > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  a.q = q;
  a.k = k;
  a.v = v;
  a.decay = decay;
  a.cu = cu;
  a.slot_in = slot_in;
  a.slot_out = slot_out;
  a.states = states;
  a.o = o;
  a.err = err;
  a.T = p->T;
  a.N = p->N;
  a.HV = p->HV;
  a.G = p->HV / p->H;
  a.slots = p->slots;
  a.scale = p->scale;
  prof_begin(K_LA_STEP, stream);
  cudaError_t e;
  switch (p->dtype) {
    case GDN_BF16: e = launch_la_step<__nv_bfloat16>(a, heads, stream); break;
    case GDN_FP16: e = launch_la_step<__half>(a, heads, stream); break;
    default: e = launch_la_step<float>(a, heads, stream); break;
  }
  prof_end(K_LA_STEP, stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
