// gdn_step.cu -- the recurrent form of the gated delta rule on a pool of states, for generation
// (one decay per value head: GDN; one per key channel: KDA).
//
// Per token of a sequence and value head, with S the 128 x 128 FP32 state (rows: key channels):
//   S' = Diag(a) S,  u = S'^T k^,  d = beta (v - u),  S = S' + k^ d^T,  o = scale S^T q^
// and o needs no second pass over S: S^T q^ = S'^T q^ + (k^.q^) d, so u and S'^T q^ are summed together.
// The norms enter as scalars: k^ = rk k, q^ = rq q.
//
// The columns of S are independent given k^ and q^, so a warp owns 16 columns of one head's state,
// with no other warp to wait for: lane (r, c), r = lane / 4, c = lane % 4, holds the columns 4c .. 4c+3
// of the rows 8r .. 8r+7 and 64+8r .. 64+8r+7 (64 registers).  A load of the warp covers 64 contiguous bytes
// of 8 rows.  The state is read once and stays in registers over all tokens of the sequence.
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_prof.h"

namespace gdn {

constexpr int ST_WARPS = 2;            // warps per CTA
constexpr int ST_COLS = 16;            // columns of a warp
constexpr int ST_PARTS = D / ST_COLS;  // warps per (sequence, head)
constexpr float ST_EPS = 1e-6f;        // under the root of the l2 norm

struct StepArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const int* cu;
  const int* slot_in;
  const int* slot_out;
  float* states;
  void* o;
  int* err;
  int64_t T, qs, ks, vs;
  int N, H, HV, G, slots, l2norm;
  float scale;
};

// bounds of sequence n's tokens; false (and the error word) where they are none
__device__ __forceinline__ bool sequence_bounds(const int* cu, int n, int64_t T, int* t0, int* t1) {
  if (!cu) {
    *t0 = n;
    *t1 = n + 1;
    return true;
  }
  *t0 = cu[n];
  *t1 = cu[n + 1];
  return *t0 >= 0 && *t1 >= *t0 && *t1 <= T;
}

template <typename E, bool KDA>
__global__ void __launch_bounds__(ST_WARPS * 32) step_kernel(const StepArgs a) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int64_t item = (int64_t)blockIdx.x * ST_WARPS + (threadIdx.x >> 5);
  const int part = (int)(item % ST_PARTS);
  const int h = (int)(item / ST_PARTS % a.HV);
  const int64_t n = item / ST_PARTS / a.HV;
  if (n >= a.N) return;
  int t0, t1;
  if (!sequence_bounds(a.cu, (int)n, a.T, &t0, &t1)) {
    if (lane == 0) *a.err = ST_DEVICE;
    return;
  }
  if (t0 == t1) return;
  const int from = a.slot_in ? a.slot_in[n] : (int)n;
  if (from < -1 || from >= a.slots) {
    if (lane == 0) *a.err = ST_DEVICE;
    return;
  }
  // element offset of this lane's first value within a slot
  const int64_t slot_elems = (int64_t)a.HV * STATE_F32;
  const int64_t at = (int64_t)h * STATE_F32 + r * 8 * D + part * ST_COLS + c * 4;
  float4 S[16];
  if (from >= 0) {
    const float* p = a.states + from * slot_elems + at;
#pragma unroll
    for (int j = 0; j < 16; ++j) S[j] = *reinterpret_cast<const float4*>(p + ((j & 7) + (j >> 3) * 64) * D);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) S[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int hq = h / a.G;
  const E* qp = static_cast<const E*>(a.q) + hq * D + r * 8;
  const E* kp = static_cast<const E*>(a.k) + hq * D + r * 8;
  // after the sums below, lanes with bit 4 clear hold u and those with it set S'^T q^, of this column
  const int own = c * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
  const E* vp = static_cast<const E*>(a.v) + h * D + part * ST_COLS + own;
  E* op = static_cast<E*>(a.o) + (int64_t)h * D + part * ST_COLS + own;
  for (int t = t0; t < t1; ++t) {
    float k[16], q[16];
    {
      Raw8<E> raw[4];
      raw[0].load(kp + t * a.ks);
      raw[1].load(kp + t * a.ks + 64);
      raw[2].load(qp + t * a.qs);
      raw[3].load(qp + t * a.qs + 64);
      float x[8];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        raw[m].get(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) k[m * 8 + j] = x[j];
        raw[2 + m].get(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[m * 8 + j] = x[j];
      }
    }
    const float v = to_f32(vp[t * a.vs]);
    const float beta = a.beta[(int64_t)t * a.HV + h];
    if (KDA) {
      const float* gp = a.g + ((int64_t)t * a.HV + h) * D + r * 8;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float e = expf(gp[(j & 7) + (j >> 3) * 64]);
        S[j].x *= e;
        S[j].y *= e;
        S[j].z *= e;
        S[j].w *= e;
      }
    } else {
      const float e = expf(a.g[(int64_t)t * a.HV + h]);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        S[j].x *= e;
        S[j].y *= e;
        S[j].z *= e;
        S[j].w *= e;
      }
    }
    float s[8], kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      s[0] += S[j].x * k[j];
      s[1] += S[j].y * k[j];
      s[2] += S[j].z * k[j];
      s[3] += S[j].w * k[j];
      s[4] += S[j].x * q[j];
      s[5] += S[j].y * q[j];
      s[6] += S[j].z * q[j];
      s[7] += S[j].w * q[j];
      kk += k[j] * k[j];
      qq += q[j] * q[j];
      kq += k[j] * q[j];
    }
    // sums over the 8 row lanes; the 8 column sums are spread over them on the way
#pragma unroll
    for (int x = 4; x <= 16; x <<= 1) {
      kk += __shfl_xor_sync(~0u, kk, x);
      qq += __shfl_xor_sync(~0u, qq, x);
      kq += __shfl_xor_sync(~0u, kq, x);
    }
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float w[4], y[2], sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float keep = b4 ? s[4 + i] : s[i], give = b4 ? s[i] : s[4 + i];
      w[i] = keep + __shfl_xor_sync(~0u, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float keep = b3 ? w[2 + i] : w[i], give = b3 ? w[i] : w[2 + i];
      y[i] = keep + __shfl_xor_sync(~0u, give, 8);
    }
    {
      const float keep = b2 ? y[1] : y[0], give = b2 ? y[0] : y[1];
      sum = keep + __shfl_xor_sync(~0u, give, 4);
    }
    const float rk = a.l2norm ? rsqrtf(kk + ST_EPS) : 1.f, rq = a.l2norm ? rsqrtf(qq + ST_EPS) : 1.f;
    const float d = beta * (v - rk * sum);   // of column `own`, in the lanes with bit 4 clear
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = rk * __shfl_sync(~0u, d, c + ((i >> 1) << 3) + ((i & 1) << 2));
    const float dq = __shfl_xor_sync(~0u, d, 16);
    if (b4) op[(int64_t)t * a.HV * D] = from_f32<E>(a.scale * rq * (sum + kq * rk * dq));
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      S[j].x += k[j] * f[0];
      S[j].y += k[j] * f[1];
      S[j].z += k[j] * f[2];
      S[j].w += k[j] * f[3];
    }
    const int to = a.slot_out ? a.slot_out[t] : t == t1 - 1 ? from : -1;
    if (to >= a.slots || to < -1) {
      if (lane == 0) *a.err = ST_DEVICE;
    } else if (to >= 0) {
      float* p = a.states + to * slot_elems + at;
#pragma unroll
      for (int j = 0; j < 16; ++j) *reinterpret_cast<float4*>(p + ((j & 7) + (j >> 3) * 64) * D) = S[j];
    }
  }
}

static bool step_stride(int64_t* s, int heads, int esize) {
  if (*s == 0) *s = (int64_t)heads * D;
  return *s >= (int64_t)heads * D && *s * esize % 16 == 0;
}

template <bool KDA>
static gdn_status run_step(const gdn_step_problem* p, const void* q, const void* k, const void* v, const float* g,
                           const float* beta, const int32_t* cu, const int32_t* slot_in, const int32_t* slot_out,
                           float* states, void* o, int32_t* err, cudaStream_t stream) {
  if (!p || p->T < 0 || p->N < 0 || p->H < 1 || p->HV < 1 || p->slots < 0) return GDN_ERR_INVALID_ARG;
  if (p->dk != D || p->dv != D || p->HV % p->H != 0 || p->T > (int64_t)INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
  if (p->dtype != GDN_BF16 && p->dtype != GDN_FP16 && p->dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
  if (!cu && p->T != p->N) return GDN_ERR_INVALID_ARG;
  if (!slot_in && p->slots < p->N) return GDN_ERR_INVALID_ARG;
  StepArgs a;
  a.qs = p->q_stride;
  a.ks = p->k_stride;
  a.vs = p->v_stride;
  const int es = elem_bytes(p->dtype);
  if (!step_stride(&a.qs, p->H, es) || !step_stride(&a.ks, p->H, es) || !step_stride(&a.vs, p->HV, es))
    return GDN_ERR_INVALID_ARG;
  if (!err) return GDN_ERR_INVALID_ARG;
  if (p->T == 0 || p->N == 0) return GDN_OK;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) || !aligned16(o) ||
      (p->slots > 0 && !aligned16(states)))
    return GDN_ERR_INVALID_ARG;
  const int64_t warps = (int64_t)p->N * p->HV * ST_PARTS;
  const int64_t ctas = (warps + ST_WARPS - 1) / ST_WARPS;
  if (ctas > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.cu = cu;
  a.slot_in = slot_in;
  a.slot_out = slot_out;
  a.states = states;
  a.o = o;
  a.err = err;
  a.T = p->T;
  a.N = p->N;
  a.H = p->H;
  a.HV = p->HV;
  a.G = p->HV / p->H;
  a.slots = p->slots;
  a.l2norm = p->l2norm;
  a.scale = p->scale;
  const int id = KDA ? K_KDA_STEP : K_STEP;
  prof_begin(id, stream);
  switch (p->dtype) {
    case GDN_BF16: step_kernel<__nv_bfloat16, KDA><<<(unsigned)ctas, ST_WARPS * 32, 0, stream>>>(a); break;
    case GDN_FP16: step_kernel<__half, KDA><<<(unsigned)ctas, ST_WARPS * 32, 0, stream>>>(a); break;
    default: step_kernel<float, KDA><<<(unsigned)ctas, ST_WARPS * 32, 0, stream>>>(a); break;
  }
  prof_end(id, stream);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_step(const gdn_step_problem* prob, const void* q, const void* k, const void* v, const float* g,
                    const float* beta, const int32_t* cu_dev, const int32_t* slot_in, const int32_t* slot_out,
                    float* states, void* o, int32_t* dev_err, struct CUstream_st* stream) {
  return run_step<false>(prob, q, k, v, g, beta, cu_dev, slot_in, slot_out, states, o, dev_err, stream);
}

gdn_status gdn_kda_step(const gdn_step_problem* prob, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, const int32_t* cu_dev, const int32_t* slot_in, const int32_t* slot_out,
                        float* states, void* o, int32_t* dev_err, struct CUstream_st* stream) {
  return run_step<true>(prob, q, k, v, g, beta, cu_dev, slot_in, slot_out, states, o, dev_err, stream);
}

}  // extern "C"
