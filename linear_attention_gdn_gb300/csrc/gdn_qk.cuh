// gdn_qk.cuh -- the norm of q and k per head with the position rotation: arguments and device pieces
// that the forward (gdn_qk.cu) and the backward (gdn_qk_bwd.cu) share.
//
// The rotation's angle p f is counted in turns as a 64-bit fixed-point fraction: the turns per position
// f / 2 pi are converted from FP64 once per CTA, and p times that, modulo 2^64, keeps its fraction exactly.
// cos and sin are FP32 of an FP32 angle within half a turn, whatever p is.
#pragma once
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_elem.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr int QK_THREADS = 256;
constexpr int QK_MAXD = 512;       // any layout
constexpr int QK_FAST_MAXD = 256;  // rows of 8-value vectors
constexpr int QK_BATCH = 4;        // rows a thread has requested together
constexpr int QK_MAX_TILE = 8;     // tokens per tile, at most
constexpr int QK_CTAS = 8;         // CTAs per SM, at most
constexpr int QK_BWD_CTAS = 2;     // of the fast backward kernel
constexpr int QK_ROW_WARPS = 4;    // rows a CTA of the other kernels has at a time

struct QkArgs {
  const void* x[2];      // q, k
  const void* in[2];     // backward: the outputs' gradients
  void* out[2];          // forward: the outputs; backward: dq, dk
  const float* w[2];
  float* part;           // backward: [CTAs][2][D] partial sums of dwq, dwk, or null
  const double* freq;
  const int* pos;
  const int* cu;
  int64_t xt[2], xh[2];  // strides of x (backward: and of out)
  int64_t yt[2], yh[2];  // strides of out (backward: of in)
  int64_t T;
  int N, heads[2], D, rot, half_layout;
  int normed;            // 0: r = 1
  float share, eps;      // r = 1 / sqrt(share x.x + eps)
  float mscale;
  // the fast kernels' work: tiles of `tile` tokens; per token items[0] + items[1] runs of `run` heads
  int tile, run, items[2];
  int64_t tiles;
};

// turns per position as a fraction of 2^64
__device__ __forceinline__ uint64_t turn_step(double f) {
  const double t = f * 0.15915494309189533577;   // 1 / (2 pi)
  return (uint64_t)((t - floor(t)) * 18446744073709551616.0);
}
__device__ __forceinline__ void angle_cos_sin(uint64_t step, int pos, float m, float* c, float* s) {
  const uint64_t turn = step * (uint64_t)(int64_t)pos;
  const float half_turns = (float)(int)(uint32_t)(turn >> 32) * (1.f / 2147483648.f);   // [-1, 1]
  sincospif(half_turns, s, c);
  *c *= m;
  *s *= m;
}

// the position of token t; `doc` carries the document found for an earlier token
__device__ __forceinline__ int position_of(const QkArgs& a, int64_t t, int* doc) {
  if (a.pos) return a.pos[t];
  if (!a.cu) return (int)t;
  int d = *doc;
  if (d + 1 < a.N && t >= a.cu[d + 1]) {   // the last document that starts at or before t
    int lo = d + 1, hi = a.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    *doc = d = lo;
  }
  return (int)t - a.cu[d];
}

// cos and sin of a tile's tokens into shared memory, row_len values a token; past rot / 2 the
// identity.  Every thread has its own document cursor, since tokens only grow.
__device__ __forceinline__ void fill_angles(const QkArgs& a, const uint64_t* step, int64_t tile, int row_len,
                                            float* cosv, float* sinv, int* doc) {
  for (int i = threadIdx.x; i < a.tile * row_len; i += QK_THREADS) {
    const int j = i / row_len, f = i - j * row_len;
    const int64_t t = tile * a.tile + j;
    float c = 1.f, s = 0.f;
    if (t < a.T && f < a.rot / 2) angle_cos_sin(step[f], position_of(a, t, doc), a.mscale, &c, &s);
    cosv[i] = c;
    sinv[i] = s;
  }
}

// Partner values of a rotated pair, for a thread with 8 values of a row in L lanes.  In the half layout
// the partner of a 4-value block is the block half its rotated part away, in another lane: block b of
// the row goes with b + rot / 8, from the other half with b - rot / 8.
template <int L> struct HalfPartner {
  int src[2];   // lanes that hold the partners of this lane's two blocks
  bool flip;    // a partner is the other block of its lane
  __device__ __forceinline__ void setup(int rot) {
    const int lane = threadIdx.x & 31, l = lane % L, away = rot / 8;
    flip = away & 1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int b = 2 * l + s;
      const int p = b < away ? b + away : b < 2 * away ? b - away : b;
      src[s] = lane - l + p / 2;
    }
  }
  __device__ __forceinline__ uint32_t get(uint32_t first, uint32_t second, int s) const {
    // what a lane sends for block s of the receivers: its own block s, or the other one
    const uint32_t give = (s == 0) != flip ? first : second;
    return __shfl_sync(~0u, give, src[s]);
  }
  template <typename E> __device__ __forceinline__ void get(const Raw8<E>& x, Raw8<E>* p) const {
    p->u.x = get(x.u.x, x.u.z, 0);
    p->u.y = get(x.u.y, x.u.w, 0);
    p->u.z = get(x.u.x, x.u.z, 1);
    p->u.w = get(x.u.y, x.u.w, 1);
  }
  __device__ __forceinline__ float getf(float first, float second, int s) const {
    return __uint_as_float(get(__float_as_uint(first), __float_as_uint(second), s));
  }
  __device__ __forceinline__ void get(const Raw8<float>& x, Raw8<float>* p) const {
    p->a = make_float4(getf(x.a.x, x.b.x, 0), getf(x.a.y, x.b.y, 0), getf(x.a.z, x.b.z, 0), getf(x.a.w, x.b.w, 0));
    p->b = make_float4(getf(x.a.x, x.b.x, 1), getf(x.a.y, x.b.y, 1), getf(x.a.z, x.b.z, 1), getf(x.a.w, x.b.w, 1));
  }
};

// This thread's cos and signed sin of one token: y[i] = z[i] co[i] + z[partner of i] si[i].  The backward's
// rotation, by the other angle, is -si.
template <int L, bool HALF>
__device__ __forceinline__ void thread_angles(const QkArgs& a, const float* cosv, const float* sinv, int row_len,
                                              float (&co)[8], float (&si)[8]) {
  const int d0 = (threadIdx.x % L) * 8;
  if (HALF) {
    const int half = a.rot / 2;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int d = d0 + 4 * s;   // half is a multiple of 4: a block of 4 lies in one half
      if (d < a.rot) {
        const int f = d < half ? d : d - half;
        const float4 c = *reinterpret_cast<const float4*>(cosv + f), v = *reinterpret_cast<const float4*>(sinv + f);
        const float sign = d < half ? -1.f : 1.f;
        co[4 * s] = c.x; co[4 * s + 1] = c.y; co[4 * s + 2] = c.z; co[4 * s + 3] = c.w;
        si[4 * s] = sign * v.x; si[4 * s + 1] = sign * v.y; si[4 * s + 2] = sign * v.z; si[4 * s + 3] = sign * v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          co[4 * s + i] = 1.f;
          si[4 * s + i] = 0.f;
        }
      }
    }
  } else if (d0 / 2 < row_len) {
    const float4 c = *reinterpret_cast<const float4*>(cosv + d0 / 2), v = *reinterpret_cast<const float4*>(sinv + d0 / 2);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      co[2 * i] = co[2 * i + 1] = cc[i];
      si[2 * i] = -ss[i];
      si[2 * i + 1] = ss[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      co[i] = 1.f;
      si[i] = 0.f;
    }
  }
}

// the partners of a thread's 8 values; zero for values that are not rotated (an infinite neighbour
// must not meet their zero sine)
template <int L, bool HALF, typename E>
__device__ __forceinline__ void partner(const HalfPartner<L>& hp, const QkArgs& a, const Raw8<E>& x, float (&p)[8]) {
  if (HALF) {
    Raw8<E> r;
    hp.get(x, &r);
    r.get(p);
  } else {
    float v[8];
    x.get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = v[i ^ 1];
  }
  if (a.rot < a.D) {
    const int rotated = a.rot - (threadIdx.x % L) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = i < rotated ? p[i] : 0.f;
  }
}

template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int x = L / 2; x >= 1; x >>= 1) v += __shfl_xor_sync(~0u, v, x);
  return v;
}

// the 8 weights of this thread (zeros past D)
__device__ __forceinline__ void load_weights(const float* w, int d0, int D, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = d0 >= D ? 0.f : w ? w[d0 + i] : 1.f;
}

inline __host__ __device__ int angle_row(int rot) { return (rot / 2 + 7) / 8 * 8; }
// shared memory of the fast kernels: the turn steps, then two buffers of cos and sin rows
inline __host__ __device__ size_t angle_smem(int rot, int tile) {
  return (size_t)angle_row(rot) * 8 + 2 * 2 * (size_t)tile * angle_row(rot) * 4;
}

// --- gdn_qk_bwd.cu ---
void launch_qk_bwd(const QkArgs& a, int dtype, bool fast, int ctas, float* dwq, float* dwk, cudaStream_t s);

}  // namespace gdn
