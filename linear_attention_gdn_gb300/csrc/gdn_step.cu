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

#include <mutex>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_prof.h"

namespace gdn {

constexpr int ST_WARPS = 2;            // warps per CTA
constexpr int ST_COLS = 16;            // columns of a warp
constexpr int ST_PARTS = D / ST_COLS;  // warps per (sequence, head)
constexpr int ST_LONG = 12;            // tokens a sequence from which on four are taken at a time
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
// A CTA of STB_WARPS warps has 16 columns a warp of one (sequence, head).  The vectors that all columns share are
// worked out once a CTA: a phase is STB_WARPS blocks, each prepared by one warp into shared memory, then taken by all
// warps without a wait. A block ends early where a state has to be written.
constexpr int STB_WARPS = 4;
constexpr int STB_TOKENS = 4;                        // tokens of a block
constexpr int STB_COLS = STB_WARPS * ST_COLS;        // columns of a CTA
constexpr int STB_PARTS = D / STB_COLS;
// sums and scalars of a block
constexpr int STB_L = 0, STB_M = 6, STB_KK = 16, STB_QQ = 20, STB_BETA = 24, STB_SCALARS = 28;

struct StepBlock {
  float kt[STB_TOKENS][D], qt[STB_TOKENS][D];   // E(0,t) k_t, E(0,t) q_t
  float kh[STB_TOKENS][D];                      // E(t,4) k_t
  float decay[D];                               // E(0,4)
  float v[STB_TOKENS][STB_COLS];
  float scalars[STB_SCALARS];                   // the pair sums, then rk, rq scale, beta
};

// One warp prepares the block of `len` tokens from t on; tokens past len change nothing.
template <typename E, bool KDA>
__device__ __forceinline__ void prepare_block(const StepArgs& a, int h, int part, int t, int len, StepBlock* blk) {
  const int lane = threadIdx.x & 31, hq = h / a.G;
  float k[4][4], q[4][4], dec[4][4], v[4][STB_COLS / 32], beta = 0.f;
  RawV<E, 4> rk[4], rq[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t ts = t + s;
    if (s < len) {
      rk[s].load(static_cast<const E*>(a.k) + ts * a.ks + hq * D + lane * 4);
      rq[s].load(static_cast<const E*>(a.q) + ts * a.qs + hq * D + lane * 4);
      const E* vp = static_cast<const E*>(a.v) + ts * a.vs + h * D + part * STB_COLS + lane;
#pragma unroll
      for (int i = 0; i < STB_COLS / 32; ++i) v[s][i] = to_f32(vp[32 * i]);
      if (KDA) {
        const float4 g = *reinterpret_cast<const float4*>(a.g + (ts * a.HV + h) * D + lane * 4);
        dec[s][0] = g.x; dec[s][1] = g.y; dec[s][2] = g.z; dec[s][3] = g.w;
      } else {
        dec[s][0] = a.g[ts * a.HV + h];
      }
    } else {
      rk[s].zero();
      rq[s].zero();
#pragma unroll
      for (int i = 0; i < STB_COLS / 32; ++i) v[s][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) dec[s][i] = 0.f;
    }
  }
  if (lane >= STB_BETA && lane - STB_BETA < len) beta = a.beta[(int64_t)(t + lane - STB_BETA) * a.HV + h];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    rk[s].get(k[s]);
    rq[s].get(q[s]);
    if (KDA) {
#pragma unroll
      for (int i = 0; i < 4; ++i) dec[s][i] = expf(dec[s][i]);
    } else {
      dec[s][0] = expf(dec[s][0]);
      dec[s][1] = dec[s][2] = dec[s][3] = dec[s][0];
    }
#pragma unroll
    for (int i = 0; i < STB_COLS / 32; ++i) blk->v[s][lane + 32 * i] = v[s][i];
  }
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

template <typename E, bool KDA>
__global__ void __launch_bounds__(STB_WARPS * 32, 4) step_block_kernel(const StepArgs a) {
  extern __shared__ __align__(16) uint8_t step_smem[];
  StepBlock* blocks = reinterpret_cast<StepBlock*>(step_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  const int part = blockIdx.x % STB_PARTS, h = blockIdx.x / STB_PARTS % a.HV, n = blockIdx.x / STB_PARTS / a.HV;
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
  // This lane has 4 columns of the rows 32 m + 4 r + 0..3, m < 4, as pairs of rows: S[2 m + i][col] holds the rows
  // 32 m + 4 r + 2 i and the next
  const int64_t slot_elems = (int64_t)a.HV * STATE_F32;
  const int col0 = part * STB_COLS + warp * ST_COLS + c * 4;
  const int64_t at = (int64_t)h * STATE_F32 + r * 4 * D + col0;
  float2 S[8][4];
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (from >= 0) {
      const float* p = a.states + from * slot_elems + at + ((m >> 1) * 32 + (m & 1) * 2) * D;
      x = *reinterpret_cast<const float4*>(p);
      y = *reinterpret_cast<const float4*>(p + D);
    }
    S[m][0] = make_float2(x.x, y.x);
    S[m][1] = make_float2(x.y, y.y);
    S[m][2] = make_float2(x.z, y.z);
    S[m][3] = make_float2(x.w, y.w);
  }
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  const int own = c * 4 + (b3 ? 2 : 0) + (b2 ? 1 : 0);   // this lane's column of the sums, within the warp's
  E* op = static_cast<E*>(a.o) + (int64_t)h * D + part * STB_COLS + warp * ST_COLS + own;

  int t = t0;
  while (t < t1) {
    // the phase's blocks: up to 4 tokens each, a state that is wanted only at a block's end
    const int look = t + lane;
    const int wants = look >= t1 ? -1 : a.slot_out ? a.slot_out[look] : look == t1 - 1 ? from : -1;
    const unsigned cuts = __ballot_sync(~0u, wants != -1);
    auto length = [&](int pos) {
      const int len = min(STB_TOKENS, t1 - t - pos), cut = __ffs(pos < 32 ? cuts >> pos : 0u);
      return cut ? min(len, cut) : len;
    };
    int pos = 0;
    for (int b = 0; b < warp; ++b) pos += length(pos);
    __syncthreads();   // the last phase's blocks have been read
    {
      const int len = length(pos);
      if (len > 0) prepare_block<E, KDA>(a, h, part, t + pos, len, blocks + warp);
    }
    __syncthreads();
    pos = 0;
    for (int b = 0; b < STB_WARPS; ++b) {
      const int len = length(pos);
      if (len <= 0) break;
      const StepBlock& blk = blocks[b];
      // S0^T with the vectors of two tokens at a time: sum[token][u, o][column]
      float sum[4][2][4];
#pragma unroll
      for (int two = 0; two < 2; ++two) {
        float2 acc[2][2][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i >> 3][i >> 2 & 1][i & 3] = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
              const float* src = kind ? blk.qt[2 * two + i] : blk.kt[2 * two + i];
              const float4 x = *reinterpret_cast<const float4*>(src + 32 * m + 4 * r);
#pragma unroll
              for (int col = 0; col < 4; ++col) {
                acc[i][kind][col] = __ffma2_rn(S[2 * m][col], make_float2(x.x, x.y), acc[i][kind][col]);
                acc[i][kind][col] = __ffma2_rn(S[2 * m + 1][col], make_float2(x.z, x.w), acc[i][kind][col]);
              }
            }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = acc[i >> 3][i >> 2 & 1][i & 3];
          sum[2 * two + (i >> 3)][i >> 2 & 1][i & 3] = x.x + x.y;
        }
      }
      // over the 8 row lanes: a lane ends with column `own`, of u (bit 4 clear) or o (set), all four tokens
      float y[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float w[4], z[2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = (b4 ? sum[s][1][i] : sum[s][0][i]) + __shfl_xor_sync(~0u, b4 ? sum[s][0][i] : sum[s][1][i], 16);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          z[i] = (b3 ? w[2 + i] : w[i]) + __shfl_xor_sync(~0u, b3 ? w[i] : w[2 + i], 8);
        y[s] = (b2 ? z[1] : z[0]) + __shfl_xor_sync(~0u, b2 ? z[0] : z[1], 4);
      }
      float sc[STB_SCALARS];
#pragma unroll
      for (int i = 0; i < STB_SCALARS / 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(blk.scalars + 4 * i);
        sc[4 * i] = x.x; sc[4 * i + 1] = x.y; sc[4 * i + 2] = x.z; sc[4 * i + 3] = x.w;
      }
      float e[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float u = y[s];
#pragma unroll
        for (int i = 0; i < s; ++i) u = fmaf(sc[STB_L + s * (s - 1) / 2 + i], e[i], u);
        const float rk = sc[STB_KK + s];
        e[s] = rk * sc[STB_BETA + s] * fmaf(-rk, u, blk.v[s][warp * ST_COLS + own]);
      }
      float2 f[4][4];   // e of this lane's columns, twice each
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float mine = __shfl_sync(~0u, e[s], lane & 15);   // the u lane's, in the o lane too
#pragma unroll
        for (int col = 0; col < 4; ++col) {
          const float x = __shfl_sync(~0u, mine, c + ((col >> 1) << 3) + ((col & 1) << 2));
          f[s][col] = make_float2(x, x);
        }
        e[s] = mine;
      }
      if (b4) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          float o = y[s];
#pragma unroll
          for (int i = 0; i <= s; ++i) o = fmaf(sc[STB_M + s * (s + 1) / 2 + i], e[i], o);
          if (s < len) op[(int64_t)(t + pos + s) * a.HV * D] = from_f32<E>(sc[STB_QQ + s] * o);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float4 x = *reinterpret_cast<const float4*>(blk.decay + 32 * m + 4 * r);
#pragma unroll
        for (int col = 0; col < 4; ++col) {
          S[2 * m][col] = __fmul2_rn(S[2 * m][col], make_float2(x.x, x.y));
          S[2 * m + 1][col] = __fmul2_rn(S[2 * m + 1][col], make_float2(x.z, x.w));
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float4 k = *reinterpret_cast<const float4*>(blk.kh[s] + 32 * m + 4 * r);
#pragma unroll
          for (int col = 0; col < 4; ++col) {
            S[2 * m][col] = __ffma2_rn(make_float2(k.x, k.y), f[s][col], S[2 * m][col]);
            S[2 * m + 1][col] = __ffma2_rn(make_float2(k.z, k.w), f[s][col], S[2 * m + 1][col]);
          }
        }
      }
      pos += len;
      if (cuts >> (pos - 1) & 1) {   // (pos <= 4 STB_WARPS <= 32)
        const int to = __shfl_sync(~0u, wants, pos - 1);
        if (to < 0 || to >= a.slots) {
          if (lane == 0) *a.err = ST_DEVICE;
        } else {
          float* p = a.states + to * slot_elems + at;
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            float* row = p + ((m >> 1) * 32 + (m & 1) * 2) * D;
            *reinterpret_cast<float4*>(row) = make_float4(S[m][0].x, S[m][1].x, S[m][2].x, S[m][3].x);
            *reinterpret_cast<float4*>(row + D) = make_float4(S[m][0].y, S[m][1].y, S[m][2].y, S[m][3].y);
          }
        }
      }
    }
    t += pos;
  }
}

constexpr int STB_SMEM = STB_WARPS * (int)sizeof(StepBlock);

template <typename E, bool KDA>
static void launch_step(const StepArgs& a, bool long_rows, unsigned ctas, cudaStream_t s) {
  if (long_rows) step_block_kernel<E, KDA><<<ctas, STB_WARPS * 32, STB_SMEM, s>>>(a);
  else step_kernel<E, KDA><<<ctas, ST_WARPS * 32, 0, s>>>(a);
}

template <typename E, bool KDA> static bool allow_smem() {
  return cudaFuncSetAttribute(step_block_kernel<E, KDA>, cudaFuncAttributeMaxDynamicSharedMemorySize, STB_SMEM) ==
         cudaSuccess;
}
// once a device
static bool step_setup() {
  static std::mutex mu;
  static bool done[128] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return false;
  std::lock_guard<std::mutex> lk(mu);
  if (!done[dev])
    done[dev] = allow_smem<__nv_bfloat16, false>() && allow_smem<__half, false>() && allow_smem<float, false>() &&
                allow_smem<__nv_bfloat16, true>() && allow_smem<__half, true>() && allow_smem<float, true>();
  return done[dev];
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
  // by the mean length, all that the host knows
  const bool long_rows = p->T >= (int64_t)p->N * ST_LONG;
  const int64_t ctas = (int64_t)p->N * p->HV * (long_rows ? STB_PARTS : ST_PARTS / ST_WARPS);
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
  if (!step_setup()) return GDN_ERR_CUDA;
  const int id = KDA ? K_KDA_STEP : K_STEP;
  prof_begin(id, stream);
  switch (p->dtype) {
    case GDN_BF16: launch_step<__nv_bfloat16, KDA>(a, long_rows, (unsigned)ctas, stream); break;
    case GDN_FP16: launch_step<__half, KDA>(a, long_rows, (unsigned)ctas, stream); break;
    default: launch_step<float, KDA>(a, long_rows, (unsigned)ctas, stream); break;
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
