// gdn_step.cu -- the recurrent form of the gated delta rule on a pool of states, for generation
// (one decay per value head: GDN; one per key channel: KDA).
//
// Per token of a sequence and value head, with S the 128 x 128 FP32 state (rows: key channels):
//   S' = Diag(a) S,  u = S'^T k^,  d = beta (v - u),  S = S' + k^ d^T,  o = scale S^T q^
// and o needs no second pass over S: S^T q^ = S'^T q^ + (k^.q^) d, so u and S'^T q^ are summed together.
// The norms enter as scalars: k^ = rk k, q^ = rq q.
//
// The columns of S are independent given k^ and q^, so a warp owns 16 columns of one head's state,
// with no other warp to wait for: lane (r, c) = (lane / 4, lane % 4) holds the columns 4c .. 4c+3 of the rows
// 8r .. 8r+7 and 64+8r .. 64+8r+7 in 64 registers.  A load of the warp covers 64 contiguous bytes of 8 rows.  The
// state is read once and stays in registers over all tokens of the sequence.
//
// One token a sequence is bound by the states' bytes: 512 sequences of 48 heads move 3.24 GB in 462 us, 7.0 TB/s;
// one sequence (6.3 MB) takes 2.5 us in a graph, 4.0 called back to back, most of it the launch and two dependent loads.  Longer sequences are bound by FP32
// arithmetic, 4 multiply-adds a state value a token (step_kernel) or 3 1/4 (step_block_kernel).
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_prof.h"

namespace gdn {

constexpr int ST_WARPS = 1;            // warps per CTA
constexpr int ST_COLS = 16;            // columns of a warp
constexpr int ST_PARTS = D / ST_COLS;  // warps per (sequence, head)
constexpr int ST_FEW = 4;              // few heads: one to so many SMs
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
  int N, H, HV, G, slots, l2norm, sms;
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

// What follows the sums of one token, the same in both kernels of single tokens: e = rk d of a column from its u, and
// its output from S'^T q^ and e.
struct StepOut {
  float e, rq;
};
__device__ __forceinline__ StepOut step_column(const StepArgs& a, float kk, float qq, float u, float beta, float v) {
  const float rk = a.l2norm ? rsqrtf(kk + ST_EPS) : 1.f, rq = a.l2norm ? rsqrtf(qq + ST_EPS) : 1.f;
  return {__fmul_rn(__fmul_rn(beta, rk), __fmaf_rn(-rk, u, v)), __fmul_rn(a.scale, rq)};
}
__device__ __forceinline__ float step_output(const StepOut& x, float kq, float sum, float e) {
  return __fmul_rn(x.rq, __fmaf_rn(kq, e, sum));
}

// about one token a sequence
template <typename E, bool KDA>
__global__ void __launch_bounds__(ST_WARPS * 32) step_token_kernel(const StepArgs a) {
  chain_kernel();
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
    // even and odd rows apart, and then as step_kernel does it: the same bits
    float s[2][8], kk[2], qq[2], kq[2];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int i = j & 1;
      const float col[4] = {S[j].x, S[j].y, S[j].z, S[j].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s[i][x] = j < 2 ? __fmul_rn(col[x], k[j]) : __fmaf_rn(col[x], k[j], s[i][x]);
        s[i][4 + x] = j < 2 ? __fmul_rn(col[x], q[j]) : __fmaf_rn(col[x], q[j], s[i][4 + x]);
      }
      kk[i] = j < 2 ? __fmul_rn(k[j], k[j]) : __fmaf_rn(k[j], k[j], kk[i]);
      qq[i] = j < 2 ? __fmul_rn(q[j], q[j]) : __fmaf_rn(q[j], q[j], qq[i]);
      kq[i] = j < 2 ? __fmul_rn(k[j], q[j]) : __fmaf_rn(k[j], q[j], kq[i]);
    }
    // sums over the 8 row lanes; the 8 column sums are spread over them on the way
    float n0 = __fadd_rn(kk[0], kk[1]), n1 = __fadd_rn(qq[0], qq[1]), n2 = __fadd_rn(kq[0], kq[1]);
#pragma unroll
    for (int x = 4; x <= 16; x <<= 1) {
      n0 += __shfl_xor_sync(~0u, n0, x);
      n1 += __shfl_xor_sync(~0u, n1, x);
      n2 += __shfl_xor_sync(~0u, n2, x);
    }
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float w[4], y[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = __fadd_rn(s[0][i], s[1][i]), o = __fadd_rn(s[0][4 + i], s[1][4 + i]);
      w[i] = (b4 ? o : u) + __shfl_xor_sync(~0u, b4 ? u : o, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) y[i] = (b3 ? w[2 + i] : w[i]) + __shfl_xor_sync(~0u, b3 ? w[i] : w[2 + i], 8);
    const float sum = (b2 ? y[1] : y[0]) + __shfl_xor_sync(~0u, b2 ? y[0] : y[1], 4);
    const StepOut r1 = step_column(a, n0, n1, sum, beta, v);
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __shfl_sync(~0u, r1.e, c + ((i >> 1) << 3) + ((i & 1) << 2));
    const float e1 = __shfl_xor_sync(~0u, r1.e, 16);
    if (b4) op[(int64_t)t * a.HV * D] = from_f32<E>(step_output(r1, n2, sum, e1));
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      S[j].x = __fmaf_rn(k[j], f[0], S[j].x);
      S[j].y = __fmaf_rn(k[j], f[1], S[j].y);
      S[j].z = __fmaf_rn(k[j], f[2], S[j].z);
      S[j].w = __fmaf_rn(k[j], f[3], S[j].w);
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

// The layout of a warp with ROWL row lanes: lane (r, c) = (lane / COLL, lane % COLL) holds the columns 4c .. 4c+3 of ROWS
// rows, in GROUPS runs of 8 neighbouring ones: 8 r + 64 m + 0 .. 7.  8 row lanes (16 rows a lane, 16 columns a warp) need the
// fewest instructions in all, 16 (8 rows, 8 columns) fewer in a warp, whose chain from token to token is all there is to
// wait for where warps are few.
template <int ROWL> struct StepLayout {
  static constexpr int COLL = 32 / ROWL, COLS = 4 * COLL, PARTS = D / COLS, ROWS = D / ROWL, GROUPS = ROWS / 8;
  static constexpr int PAIRS = ROWS / 2;
  // the first row, within a lane's, of the pair p
  static __device__ __forceinline__ int row(int p) { return p % 4 * 2 + p / 4 * 64; }
};

// what a lane needs of one token
template <typename E, bool KDA, int ROWL> struct StepToken {
  using L = StepLayout<ROWL>;
  Raw8<E> k[L::GROUPS], q[L::GROUPS];   // of its rows
  float4 g[KDA ? L::ROWS / 4 : 1];
  float beta;
  E v;                  // of its column of the sums
  int to;
};

// a few tokens: the next one's rows are requested a token ahead, and rows lie in pairs for the paired FP32 instructions
// BUSY: registers for 12 and 16 warps an SM (64 sequences of 8 tokens 142 us with one decay a channel and 117 with one a
// head; left to the compiler 177 and 125), where there are so many warps.
template <typename E, bool KDA, int ROWL, bool BUSY>
__global__ void __launch_bounds__(32, !BUSY ? 1 : KDA || sizeof(E) == 4 ? 12 : 16) step_kernel(const StepArgs a) {
  chain_kernel();
  using L = StepLayout<ROWL>;
  using Token = StepToken<E, KDA, ROWL>;
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
  // element offset of this lane's first value within a slot
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
  // after the sums, lanes with bit 4 clear hold u and those with it set S'^T q^, of this column
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  const int own = part * L::COLS + c * 4 + (b3 ? 2 : 0) + (b2 ? 1 : 0);
  const bool writer = b4 && (lane & 3) < L::COLL;   // (further row lanes have copies of the sums)
  const int hq = h / a.G;
  auto request = [&](int64_t t, Token* x) {
    const E* kp = static_cast<const E*>(a.k) + t * a.ks + hq * D + r * 8;
    const E* qp = static_cast<const E*>(a.q) + t * a.qs + hq * D + r * 8;
#pragma unroll
    for (int m = 0; m < L::GROUPS; ++m) {
      x->k[m].load(kp + 64 * m);
      x->q[m].load(qp + 64 * m);
    }
    if constexpr (KDA) {
      const float4* g = reinterpret_cast<const float4*>(a.g + (t * a.HV + h) * D + r * 8);
#pragma unroll
      for (int m = 0; m < L::ROWS / 4; ++m) x->g[m] = g[(m & 1) + (m >> 1) * 16];
    } else {
      x->g[0].x = a.g[t * a.HV + h];
    }
    x->beta = a.beta[t * a.HV + h];
    x->v = static_cast<const E*>(a.v)[t * a.vs + h * D + own];
    x->to = a.slot_out ? a.slot_out[t] : t == t1 - 1 ? from : -1;
  };
  Token x;
  request(t0, &x);
  E* op = static_cast<E*>(a.o) + ((int64_t)t0 * a.HV + h) * D + own;
  for (int t = t0; t < t1; ++t, op += (int64_t)a.HV * D) {
    // decay: not by the fast exponential, whose values just below one are 0.2 to 0.4 last places too low on average: that adds up
    // over the tokens (256 of them: states 4.0e-7 of their columns' size from FP64, with this 1.4e-7, as with NumPy's FP32
    // exponential; 586 ragged and 37 single tokens of the per-channel rule 105.7 and 25.9 us with it, with this 108.1 and
    // 26.7; one decay a head within 1 %)
    if constexpr (KDA) {
#pragma unroll
      for (int j = 0; j < L::PAIRS; ++j) {
        const float4 g = x.g[j >> 1];
        const float2 e = j & 1 ? make_float2(expf(g.z), expf(g.w)) : make_float2(expf(g.x), expf(g.y));
#pragma unroll
        for (int i = 0; i < 4; ++i) S[j][i] = __fmul2_rn(S[j][i], e);
      }
    } else {
      const float e = expf(x.g[0].x);
#pragma unroll
      for (int j = 0; j < 4 * L::PAIRS; ++j) S[j >> 2][j & 3] = __fmul2_rn(S[j >> 2][j & 3], make_float2(e, e));
    }
    float2 k[L::PAIRS], s[2][4];
    float2 kk = make_float2(0.f, 0.f), qq = kk, kq = kk;
#pragma unroll
    for (int m = 0; m < L::GROUPS; ++m) {
      float kf[8], qf[8];
      x.k[m].get(kf);
      x.q[m].get(qf);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = 4 * m + j;
        k[p] = make_float2(kf[2 * j], kf[2 * j + 1]);
        const float2 q = make_float2(qf[2 * j], qf[2 * j + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[0][i] = p ? __ffma2_rn(S[p][i], k[p], s[0][i]) : __fmul2_rn(S[p][i], k[p]);
          s[1][i] = p ? __ffma2_rn(S[p][i], q, s[1][i]) : __fmul2_rn(S[p][i], q);
        }
        kk = __ffma2_rn(k[p], k[p], kk);
        qq = __ffma2_rn(q, q, qq);
        kq = __ffma2_rn(k[p], q, kq);
      }
    }
    const float beta = x.beta, v = to_f32(x.v);
    const int to = x.to;
    if (t + 1 < t1) request(t + 1, &x);
    // sums over the 8 row lanes; the 8 column sums are spread over them on the way
    float n0 = kk.x + kk.y, n1 = qq.x + qq.y, n2 = kq.x + kq.y;
#pragma unroll
    for (int d = L::COLL; d <= 16; d <<= 1) {
      n0 += __shfl_xor_sync(~0u, n0, d);
      n1 += __shfl_xor_sync(~0u, n1, d);
      n2 += __shfl_xor_sync(~0u, n2, d);
    }
    float w[4], y[2], sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = s[0][i].x + s[0][i].y, o = s[1][i].x + s[1][i].y;
      w[i] = (b4 ? o : u) + __shfl_xor_sync(~0u, b4 ? u : o, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) y[i] = (b3 ? w[2 + i] : w[i]) + __shfl_xor_sync(~0u, b3 ? w[i] : w[2 + i], 8);
    sum = (b2 ? y[1] : y[0]) + __shfl_xor_sync(~0u, b2 ? y[0] : y[1], 4);
#pragma unroll
    for (int d = L::COLL; d < 4; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
    const StepOut r1 = step_column(a, n0, n1, sum, beta, v);
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = __shfl_sync(~0u, r1.e, c + ((i >> 1) << 3) + ((i & 1) << 2));
      f[i] = make_float2(e, e);
    }
    const float e1 = __shfl_xor_sync(~0u, r1.e, 16);
    if (writer) *op = from_f32<E>(step_output(r1, n2, sum, e1));
#pragma unroll
    for (int j = 0; j < 4 * L::PAIRS; ++j) S[j >> 2][j & 3] = __ffma2_rn(k[j >> 2], f[j & 3], S[j >> 2][j & 3]);
    if (to >= a.slots || to < -1) {
      if (lane == 0) *a.err = ST_DEVICE;
    } else if (to >= 0) {
      float* p = a.states + to * slot_elems + at;
#pragma unroll
      for (int j = 0; j < L::PAIRS; ++j) {
        float* row = p + L::row(j) * D;
        *reinterpret_cast<float4*>(row) = make_float4(S[j][0].x, S[j][1].x, S[j][2].x, S[j][3].x);
        *reinterpret_cast<float4*>(row + D) = make_float4(S[j][0].y, S[j][1].y, S[j][2].y, S[j][3].y);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// longer sequences: four tokens at a time
// ---------------------------------------------------------------------------
// With the state S0 before a block of tokens 1..4 and E(s, t) = a_{s+1} ... a_t (channel by channel, never a quotient, so
// decays of any steepness are exact):
//   u_t = S0^T (E(0,t) k_t) + sum_{s<t} ((E(s,t) k_s) . k_t) e_s,   e_t = rk_t beta_t (v_t - rk_t u_t)
//   o_t = scale rq_t (S0^T (E(0,t) q_t) + sum_{s<=t} ((E(s,t) k_s) . q_t) e_s)
//   S   = Diag(E(0,4)) S0 + sum_s (E(s,4) k_s) e_s^T
// (k, q without their norms rk, rq).  All products with S0 are independent of the chain over the tokens, which is left
// with four values a column; and S is scaled once in four tokens.
//
// A warp owns CPL columns of each of 32 / ROWL lanes c = lane % (32 / ROWL), and lane r = lane / (32 / ROWL) of them the rows
// 4 ROWL m + 4 r + 0..3 for all m, as pairs of rows, so that what it reads of the shared vectors is used CPL times and in
// pairs as it lies.  The vectors that all columns share are worked out once a CTA: a phase is STB_WARPS blocks, each
// prepared by one warp into shared memory, then taken by all warps without a wait, while the next phase's rows are copied
// in.  A block ends early where a state has to be written.
//
// Many heads: 32 columns a warp (8 row lanes of 8 columns, 128 registers of state), a head a CTA, whose warps prepare
// and then take.  Few heads, for which the chain from block to block is all: 8 columns a warp (16 row lanes of 4), a quarter of a
// head a CTA, and the next phase is prepared by STB_WARPS further warps meanwhile (BESIDE; one sequence of 160 tokens
// and 4 heads 39 us, token by token 48).
constexpr int STB_MIN_TOKENS = 24;      // a sequence, on average
constexpr int STB_MIN_FEW = 32;         // where heads are few
constexpr int STB_MIN_FULL = 12;        // and where tokens times heads are as many as
constexpr int64_t STB_FULL = 12288;
constexpr int STB_WARPS = 4;
constexpr int STB_TOKENS = 4;   // tokens of a block
// sums and scalars of a block
constexpr int STB_L = 0, STB_M = 6, STB_KK = 16, STB_QQ = 20, STB_BETA = 24, STB_SCALARS = 28;

template <int ROWL, int CPL> struct BlockLayout {
  static constexpr int COLL = 32 / ROWL, COLS = CPL * COLL, PARTS = D / (STB_WARPS * COLS);   // PARTS: CTAs of a head
  static constexpr int APART = 4 * ROWL, RUNS = D / APART;
  static constexpr int E_BYTES = STB_TOKENS * COLS * (int)sizeof(float2);
};

struct StepBlock {
  float kt[STB_TOKENS][D], qt[STB_TOKENS][D];   // E(0,t) k_t, E(0,t) q_t
  float kh[STB_TOKENS][D];                      // E(t,4) k_t
  float decay[D];                               // E(0,4)
  float v[STB_TOKENS][D];
  float scalars[STB_SCALARS];                   // the pair sums, then rk, rq scale, beta
};

// The rows of a phase's tokens as they lie in memory (one FP32 g a token, or one a channel).
template <typename E, bool KDA> struct alignas(16) StepRaw {
  static constexpr int TOKENS = STB_WARPS * STB_TOKENS;
  E k[TOKENS][D], q[TOKENS][D], v[TOKENS][D];
  float g[TOKENS][KDA ? D : 1];
  float beta[TOKENS];
};
__device__ __forceinline__ void copy_async16(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_async4(void* smem, const void* global) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem)), "l"(global) : "memory");
}
// A warp's share of the copies: the tokens first + 4 warp + 0..3, as far as there are any
template <typename E, bool KDA>
__device__ __forceinline__ void request_rows(const StepArgs& a, int h, int first, int t1, int warp,
                                             StepRaw<E, KDA>* raw) {
  constexpr int VEC = 16 / (int)sizeof(E), ROW = D / VEC;
  const int lane = threadIdx.x & 31, hq = h / a.G;
#pragma unroll
  for (int i0 = 0; i0 < STB_TOKENS * ROW; i0 += 32) {
    const int i = i0 + lane, j = warp * STB_TOKENS + i / ROW, x = i % ROW * VEC;
    const int64_t t = first + j;
    if (t < t1) {
      copy_async16(&raw->k[j][x], static_cast<const E*>(a.k) + t * a.ks + hq * D + x);
      copy_async16(&raw->q[j][x], static_cast<const E*>(a.q) + t * a.qs + hq * D + x);
      copy_async16(&raw->v[j][x], static_cast<const E*>(a.v) + t * a.vs + h * D + x);
    }
  }
  if (KDA) {
#pragma unroll
    for (int i = 0; i < STB_TOKENS; ++i) {
      const int j = warp * STB_TOKENS + i;
      const int64_t t = first + j;
      if (t < t1) copy_async16(&raw->g[j][KDA ? lane * 4 : 0], a.g + (t * a.HV + h) * D + lane * 4);
    }
  }
  const int j = warp * STB_TOKENS + lane % STB_TOKENS;
  const int64_t t = first + j;
  if (lane < STB_TOKENS && t < t1) copy_async4(&raw->beta[j], a.beta + t * a.HV + h);
  if (!KDA && lane >= 8 && lane < 8 + STB_TOKENS && t < t1) copy_async4(&raw->g[j][0], a.g + t * a.HV + h);
}

// One warp prepares the block of `len` tokens from the phase's token j on; tokens past len change nothing.
template <typename E, bool KDA>
__device__ __forceinline__ void prepare_block(const StepArgs& a, const StepRaw<E, KDA>& raw, int j, int len,
                                              StepBlock* blk) {
  const int lane = threadIdx.x & 31;
  float k[4][4], q[4][4], dec[4][4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    RawV<E, 4> x;
    x.zero();
    if (s < len) x.load_shared(smem_u32(&raw.k[j + s][lane * 4]));
    x.get(k[s]);
    x.zero();
    if (s < len) x.load_shared(smem_u32(&raw.q[j + s][lane * 4]));
    x.get(q[s]);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) blk->v[s][lane + 32 * i] = s < len ? to_f32(raw.v[j + s][lane + 32 * i]) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dec[s][i] = s >= len ? 1.f : KDA || i == 0 ? expf(raw.g[j + s][KDA ? lane * 4 + i : 0]) : dec[s][0];
  }
  const float beta = lane >= STB_BETA && lane - STB_BETA < len ? raw.beta[j + lane - STB_BETA] : 0.f;
  float sums[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) sums[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // channels
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      float w = k[s][i];
      sums[STB_KK + s] = fmaf(w, w, sums[STB_KK + s]);
      sums[STB_QQ + s] = fmaf(q[s][i], q[s][i], sums[STB_QQ + s]);
      sums[STB_M + s * (s + 1) / 2 + s] = fmaf(w, q[s][i], sums[STB_M + s * (s + 1) / 2 + s]);
#pragma unroll
      for (int u = s + 1; u < 4; ++u) {
        w *= dec[u][i];
        sums[STB_L + u * (u - 1) / 2 + s] = fmaf(w, k[u][i], sums[STB_L + u * (u - 1) / 2 + s]);
        sums[STB_M + u * (u + 1) / 2 + s] = fmaf(w, q[u][i], sums[STB_M + u * (u + 1) / 2 + s]);
      }
      blk->kh[s][lane * 4 + i] = w;
    }
    float e = 1.f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      e *= dec[s][i];
      blk->kt[s][lane * 4 + i] = e * k[s][i];
      blk->qt[s][lane * 4 + i] = e * q[s][i];
    }
    blk->decay[lane * 4 + i] = e;
  }
  // the sums over the warp; lane i ends with sum i
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const bool upper = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? sums[half + i] : sums[i], give = upper ? sums[i] : sums[half + i];
      sums[i] = keep + __shfl_xor_sync(~0u, give, half);
    }
  }
  float x = sums[0];
  if (lane >= STB_KK && lane < STB_BETA) {
    x = a.l2norm ? rsqrtf(x + ST_EPS) : 1.f;
    if (lane >= STB_QQ) x *= a.scale;
  }
  if (lane >= STB_BETA) x = beta;
  if (lane < STB_SCALARS) blk->scalars[lane] = x;
}

// Few sequences of unlike lengths are all on the GPU at once, and an SM's time is the sum of its CTAs': so the CTAs go by
// falling length, and every second row of them over the SMs in the other direction (586 tokens in lengths
// 0 .. 160 at HV = 48: 105 us, in the sequences' own order 127 us; with the accurate exponential 108).
constexpr int STB_SORTED = 32;   // sequences that one warp ranks
__device__ __forceinline__ int balanced_place(const StepArgs& a, int place, int places) {
  if (a.N > STB_SORTED) return place;
  const int row = place / a.sms, first = row * a.sms;
  return row & 1 ? first + min(a.sms, places - first) - 1 - (place - first) : place;
}
__device__ __forceinline__ int sequence_of_rank(const StepArgs& a, int rank) {
  if (a.N > STB_SORTED || !a.cu) return rank;
  const int lane = threadIdx.x & 31, len = lane < a.N ? a.cu[lane + 1] - a.cu[lane] : INT32_MIN;
  int before = 0;   // sequences that are longer, or as long and earlier
  for (int i = 0; i < a.N; ++i) {
    const int other = __shfl_sync(~0u, len, i);
    before += other > len || (other == len && i < lane);
  }
  return __ffs(__ballot_sync(~0u, lane < a.N && before == rank)) - 1;
}

template <int ID, int THREADS> __device__ __forceinline__ void barrier() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

template <typename E, bool KDA, int ROWL, int CPL, bool BESIDE>
__global__ void __launch_bounds__(STB_WARPS * (BESIDE ? 64 : 32), 2) step_block_kernel(const StepArgs a) {
  previous_kernel_done();   // (its own dependents would take the places of balanced_place: 127 us for 105)
  using Raw = StepRaw<E, KDA>;
  extern __shared__ __align__(16) uint8_t step_smem[];
  using L = BlockLayout<ROWL, CPL>;
  constexpr int BUFFERS = BESIDE ? 2 : 1;
  StepBlock(*blocks)[STB_WARPS] = reinterpret_cast<StepBlock(*)[STB_WARPS]>(step_smem);
  Raw* raw = reinterpret_cast<Raw*>(step_smem + BUFFERS * STB_WARPS * sizeof(StepBlock));
  __shared__ int targets[BUFFERS][32];   // BESIDE: `wants` of a phase
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane / L::COLL, c = lane % L::COLL;
  const int place = balanced_place(a, blockIdx.x, gridDim.x);
  const int part = place % L::PARTS, h = place / L::PARTS % a.HV, n = sequence_of_rank(a, place / L::PARTS / a.HV);
  int t0, t1;
  if (!sequence_bounds(a.cu, n, a.T, &t0, &t1)) {
    if (threadIdx.x == 0) *a.err = ST_DEVICE;
    return;
  }
  if (t0 == t1) return;
  const int from = a.slot_in ? a.slot_in[n] : n;
  if (from < -1 || from >= a.slots) {
    if (threadIdx.x == 0) *a.err = ST_DEVICE;
    return;
  }
  int t = t0, buffer = 0;
  unsigned cuts = 0;
  // a phase's blocks: up to 4 tokens each, a state that is wanted only at a block's end
  auto length = [&](int pos) {   // (pos < 32: a phase has at most 4 * 4 tokens)
    const int len = min(STB_TOKENS, t1 - t - pos), cut = __ffs(cuts >> pos);
    return cut ? min(len, cut) : len;
  };
  auto wanted = [&](int first) {
    const int look = first + lane;
    return look >= t1 ? -1 : a.slot_out ? a.slot_out[look] : look == t1 - 1 ? from : -1;
  };
  const int w = BESIDE ? warp - STB_WARPS : warp;   // of the warps that prepare
  int wants = -1, next_wants = -1;   // where the states after a phase's tokens go: -1 nowhere
  auto begin = [&] {
    request_rows<E, KDA>(a, h, t0, t1, w, raw);
    asm volatile("cp.async.commit_group;" ::: "memory");
    next_wants = wanted(t0);
  };
  // the next phase's blocks; its number of tokens
  auto prepare = [&](StepBlock* phase) {
    wants = next_wants;
    cuts = __ballot_sync(~0u, wants != -1);
    int mine = 0, all = 0;   // where this warp's block begins
    for (int b = 0; b < STB_WARPS; ++b) {
      if (b == w) mine = all;
      all += length(all);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    barrier<1, STB_WARPS * 32>();   // the rows are there (and where the same warps take them, the last phase's blocks have been read)
    if (BESIDE && w == 0) targets[BESIDE ? buffer : 0][lane] = wants;
    if (w == 0 || mine < all) prepare_block<E, KDA>(a, *raw, mine, length(mine), phase + w);
    barrier<1, STB_WARPS * 32>();   // the blocks are there, and the rows have been read
    request_rows<E, KDA>(a, h, t + all, t1, w, raw);
    asm volatile("cp.async.commit_group;" ::: "memory");
    next_wants = wanted(t + all);
    return all;
  };
  if (BESIDE && warp >= STB_WARPS) {
    begin();
    while (t < t1) {
      const int all = prepare(blocks[buffer]);
      barrier<0, STB_WARPS * 64>();   // the phase may be taken, and the other buffer written
      t += all;
      buffer ^= 1;
    }
    return;
  }
  if (!BESIDE) begin();
  // S[2 m + i][x]: the rows 4 ROWL m + 4 r + 2 i and the next, of this lane's column x ^ turn.  With the columns in that
  // order a lane always gives the upper half of its sums away and keeps the lower.
  const int own_x = CPL == 8 ? lane >> 2 : lane >> 3, turn = own_x & (CPL - 2);
  const int column = (part * STB_WARPS + warp) * L::COLS;   // the warp's first
  const int64_t slot_elems = (int64_t)a.HV * STATE_F32;
  const int64_t at = (int64_t)h * STATE_F32 + r * 4 * D + column + c * CPL;
  float2 S[2 * L::RUNS][CPL];
#pragma unroll
  for (int m = 0; m < 2 * L::RUNS; ++m)
#pragma unroll
    for (int x = 0; x < CPL; x += 2) {   // two columns at a time
      float2 top = make_float2(0.f, 0.f), low = top;
      if (from >= 0) {
        const float* p = a.states + from * slot_elems + at + ((m >> 1) * L::APART + (m & 1) * 2) * D + (x ^ turn);
        top = *reinterpret_cast<const float2*>(p);
        low = *reinterpret_cast<const float2*>(p + D);
      }
      S[m][x] = make_float2(top.x, low.x);
      S[m][x + 1] = make_float2(top.y, low.y);
    }
  const int own = c * CPL + own_x;   // this lane's column of the sums, within the warp's
  const bool writer = lane % (L::COLL * 32 / L::COLS) < L::COLL;   // (further lanes have copies of the sums)
  E* op = static_cast<E*>(a.o) + (int64_t)h * D + column + own;
  float2(*se)[L::COLS] = reinterpret_cast<float2(*)[L::COLS]>(   // every e twice: pairs as they are used
      step_smem + BUFFERS * STB_WARPS * sizeof(StepBlock) + sizeof(Raw) + warp * L::E_BYTES);

  while (t < t1) {
    int all = 0;   // (the blocks' lengths added up once more: 107 us for 105)
    if (BESIDE) {
      barrier<0, STB_WARPS * 64>();
      wants = targets[BESIDE ? buffer : 0][lane];
      cuts = __ballot_sync(~0u, wants != -1);
    } else {
      all = prepare(blocks[0]);
    }
    const StepBlock* phase = blocks[BESIDE ? buffer : 0];
    int pos = 0;
#pragma unroll 1
    for (int b = 0; b < STB_WARPS; ++b) {
      const int len = length(pos);
      if (len <= 0) break;
      const StepBlock& blk = phase[b];
      // S0^T with a token's two vectors, summed over the row lanes: y[token][u, o] of column `own`
      float y[4][2];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float2 acc[2][CPL];
#pragma unroll
        for (int m = 0; m < L::RUNS; ++m)
#pragma unroll
          for (int kind = 0; kind < 2; ++kind) {
            const float4 x = *reinterpret_cast<const float4*>((kind ? blk.qt[s] : blk.kt[s]) + L::APART * m + 4 * r);
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
              acc[kind][i] = m ? __ffma2_rn(S[2 * m][i], make_float2(x.x, x.y), acc[kind][i])
                               : __fmul2_rn(S[0][i], make_float2(x.x, x.y));
              acc[kind][i] = __ffma2_rn(S[2 * m + 1][i], make_float2(x.z, x.w), acc[kind][i]);
            }
          }
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          float w[CPL];
#pragma unroll
          for (int i = 0; i < CPL; ++i) w[i] = acc[kind][i].x + acc[kind][i].y;
          int d = 16;
#pragma unroll
          for (int half = CPL / 2; half > 1; half >>= 1, d >>= 1)
#pragma unroll
            for (int i = 0; i < half; ++i) w[i] += __shfl_xor_sync(~0u, w[half + i], d);
          const bool upper = lane & d;
          float sum = (upper ? w[1] : w[0]) + __shfl_xor_sync(~0u, upper ? w[0] : w[1], d);
#pragma unroll
          for (d >>= 1; d >= L::COLL; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
          y[s][kind] = sum;
        }
      }
      // the chain over the tokens
      float sc[STB_SCALARS], e[4];
#pragma unroll
      for (int i = 0; i < STB_SCALARS / 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(blk.scalars + 4 * i);
        sc[4 * i] = x.x; sc[4 * i + 1] = x.y; sc[4 * i + 2] = x.z; sc[4 * i + 3] = x.w;
      }
      __syncwarp();   // the last block's e have been read
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float u = y[s][0], o = y[s][1];
#pragma unroll
        for (int i = 0; i < s; ++i) {
          u = fmaf(sc[STB_L + s * (s - 1) / 2 + i], e[i], u);
          o = fmaf(sc[STB_M + s * (s + 1) / 2 + i], e[i], o);
        }
        const float rk = sc[STB_KK + s];
        // (none from tokens past len: of infinite values their zeros would make NaN)
        e[s] = s < len ? rk * sc[STB_BETA + s] * fmaf(-rk, u, blk.v[s][column + own]) : 0.f;
        o = fmaf(sc[STB_M + s * (s + 1) / 2 + s], e[s], o);
        se[s][own] = make_float2(e[s], e[s]);
        if (s < len && writer) op[(int64_t)(t + pos + s) * a.HV * D] = from_f32<E>(sc[STB_QQ + s] * o);
      }
      __syncwarp();
#pragma unroll
      for (int m = 0; m < L::RUNS; ++m) {
        const float4 x = *reinterpret_cast<const float4*>(blk.decay + L::APART * m + 4 * r);
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
          S[2 * m][i] = __fmul2_rn(S[2 * m][i], make_float2(x.x, x.y));
          S[2 * m + 1][i] = __fmul2_rn(S[2 * m + 1][i], make_float2(x.z, x.w));
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float2 f[8];
#pragma unroll
        for (int i = 0; i < CPL; i += 2) {
          const float4 x = *reinterpret_cast<const float4*>(&se[s][c * CPL + (i ^ turn)]);
          f[i] = make_float2(x.x, x.y);
          f[i + 1] = make_float2(x.z, x.w);
        }
#pragma unroll
        for (int m = 0; m < L::RUNS; ++m) {
          const float4 k = *reinterpret_cast<const float4*>(blk.kh[s] + L::APART * m + 4 * r);
#pragma unroll
          for (int i = 0; i < CPL; ++i) {
            S[2 * m][i] = __ffma2_rn(make_float2(k.x, k.y), f[i], S[2 * m][i]);
            S[2 * m + 1][i] = __ffma2_rn(make_float2(k.z, k.w), f[i], S[2 * m + 1][i]);
          }
        }
      }
      pos += len;
      if (cuts >> (pos - 1) & 1) {
        const int to = __shfl_sync(~0u, wants, pos - 1);
        if (to < 0 || to >= a.slots) {
          if (lane == 0) *a.err = ST_DEVICE;
        } else {
#pragma unroll
          for (int m = 0; m < 2 * L::RUNS; ++m)
#pragma unroll
            for (int x = 0; x < CPL; x += 2) {
              float* p = a.states + to * slot_elems + at + ((m >> 1) * L::APART + (m & 1) * 2) * D + (x ^ turn);
              *reinterpret_cast<float2*>(p) = make_float2(S[m][x].x, S[m][x + 1].x);
              *reinterpret_cast<float2*>(p + D) = make_float2(S[m][x].y, S[m][x + 1].y);
            }
        }
      }
    }
    t += BESIDE ? pos : all;
    buffer ^= 1;
  }
}

template <typename E, bool KDA, int ROWL, int CPL, bool BESIDE>
static bool launch_blocks(const StepArgs& a, unsigned heads, cudaStream_t s) {
  using L = BlockLayout<ROWL, CPL>;
  constexpr int bytes = STB_WARPS * ((BESIDE ? 2 : 1) * (int)sizeof(StepBlock) + L::E_BYTES) + (int)sizeof(StepRaw<E, KDA>);
  const auto kernel = step_block_kernel<E, KDA, ROWL, CPL, BESIDE>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  launch_chained(kernel, heads * L::PARTS, STB_WARPS * (BESIDE ? 64 : 32), bytes, s, a);
  return true;
}

template <typename E, bool KDA> static bool launch_step(const StepArgs& a, bool blocks, unsigned heads, cudaStream_t s) {
  if (blocks) {
    if (heads > a.sms / 2) return launch_blocks<E, KDA, 8, 8, false>(a, heads, s);
    return launch_blocks<E, KDA, 16, 4, true>(a, heads, s);
  } else if (heads <= a.sms / ST_FEW) {   // single tokens, too: their bits are the same as a sequence's
    launch_chained(step_kernel<E, KDA, 16, false>, heads * StepLayout<16>::PARTS, 32, 0, s, a);
  } else if (a.T <= a.N) {
    launch_chained(step_token_kernel<E, KDA>, heads * ST_PARTS / ST_WARPS, ST_WARPS * 32, 0, s, a);
  } else if (heads <= a.sms) {
    launch_chained(step_kernel<E, KDA, 8, false>, heads * StepLayout<8>::PARTS, 32, 0, s, a);
  } else {
    launch_chained(step_kernel<E, KDA, 8, true>, heads * StepLayout<8>::PARTS, 32, 0, s, a);
  }
  return true;
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
      (p->slots > 0 && !aligned16(states)) || !on_words(cu, slot_in, slot_out, err))
    return GDN_ERR_INVALID_ARG;
  // By the sequences' heads and their mean length, which is all that the host knows of the lengths.  Few heads, for which
  // the chain from token to token is all: step_kernel with 8 columns a warp (one sequence of 64 tokens and 4 heads 20 us,
  // with 16 columns 32).  Else one token: step_token_kernel (64 sequences of 48 heads 60 us; step_kernel, with more
  // registers, 70); a few, step_kernel (64 of 8: 115 us; step_block_kernel 157); from 24 on, step_block_kernel, a CTA a
  // head, if that fills half of the SMs (3 of 48 heads, 16 tokens: 15 us against 14, 32: 22 against 24,
  // 64: 36 against 44); with fewer a quarter of a head a CTA, from 32 on (4 heads, 24 tokens: 9.5 us against 9.0, 32: 11.3
  // against 11.3, 64: 18 against 20, 160: 39 against 48; 48 heads, 64: 26 against 28); and from 12 on where warps are so many
  // that only the work counts (64 of 16: 182 us against 204, 32 of 128: 533 against 796; but 16 of 16: 58 against 57).
  const int64_t heads = (int64_t)p->N * p->HV;
  const bool blocks = heads <= sm_count() / 2 ? p->T >= (int64_t)p->N * STB_MIN_FEW
                                              : p->T >= (int64_t)p->N * STB_MIN_TOKENS ||
                                                    (p->T >= (int64_t)p->N * STB_MIN_FULL && p->T * p->HV >= STB_FULL);
  if (heads * StepLayout<16>::PARTS > INT32_MAX) return GDN_ERR_UNSUPPORTED;
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
  a.sms = sm_count();
  a.l2norm = p->l2norm;
  a.scale = p->scale;
  const int id = KDA ? K_KDA_STEP : K_STEP;
  prof_begin(id, stream);
  bool ok;
  switch (p->dtype) {
    case GDN_BF16: ok = launch_step<__nv_bfloat16, KDA>(a, blocks, (unsigned)heads, stream); break;
    case GDN_FP16: ok = launch_step<__half, KDA>(a, blocks, (unsigned)heads, stream); break;
    default: ok = launch_step<float, KDA>(a, blocks, (unsigned)heads, stream); break;
  }
  prof_end(id, stream);
  return ok && cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
