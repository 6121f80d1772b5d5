// gdn_la.cu -- linear attention with a fixed decay a per head, in chunks of L <= 128 tokens.
//
// Every result of the forward and the backward is one walk over the chunks of a document, with rows x, y, z of 128 values:
//   out_r = sum_{c seen by r} a^|r-c| (x_r . y_c) z_c + a^(tokens between) Z^T x_r,     Z <- a^L Z + sum_c a^.. y_c z_c^T
//   forward  o : x, y, z = q, k, v;     dq : dO, v, k     (r sees c <= r; Z is the state before the chunk)
//   reverse  dv: x, y, z = k, q, dO;    dk : v, dO, q     (r sees c >= r; Z is the gradient behind the chunk)
//
// A CTA walks one segment of a document for one value head.  Per chunk, on the tensor cores:
//   QK[r][c] = x_r . y_c;  Oi = x Z;  P = decayed, masked QK;  Op = P z;  dZ[z][y] = z^T (decayed y);  out = a^.. Oi + Op
// P goes back to TMEM as the left operand.  The state is FP32 in registers (thread: one row z, 64 columns y), rounded to
// BF16 once for the product with x.  The decayed y is given to the product as a sum of BF16 terms, so that the
// state keeps FP32's exactness: two terms (2^-17) where only BF16 results come of it, three (2^-25) where the state itself
// is handed out.
// Documents whose chains are too few or too long are cut into segments: la_walk without output first sums what each adds,
// la_carry_kernel turns the sums into the states they start from.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_common.cuh"
#include "gdn_la.cuh"
#include "gdn_launch.cuh"

namespace gdn {

constexpr int LA_WORK = 256;                 // threads that compute: two warpgroups, 64 columns each
constexpr int LA_THREADS = LA_WORK + 64;     // and a warp each for the MMAs and the loads
constexpr int LA_TILE = LA_CH * D * 2;       // 32 KB
constexpr int LA_STAGE = 3 * LA_TILE;
constexpr int LA_ZS = 2 * LA_STAGE;          // the state as BF16 [z][y]; then a term of the decayed y
constexpr int LA_SMEM = LA_ZS + LA_TILE + 1024;
// TMEM columns
constexpr int LT_QK = 0, LT_OI = 128, LT_OP = 256, LT_DZ = 384;
constexpr float LA_LEAST = -1e4f;   // log decays below it: nothing is left of it either, and no product is NaN

// a^n: the product's rounding error is put back, so that far powers are as exact as near ones
__device__ __forceinline__ float la_power(float g, float n) {
  const float p = g * n, e = expf(p);
  return fmaf(e, fmaf(g, n, -p), e);
}

struct LaPlace {
  int doc, index, count;   // segment `index` of the document's `count`
  int t0, t1;              // the document's tokens
};

// Segment number `want` by one warp; false if there is none.  The whole list is walked if `check`: false, too, if it does
// not have the length that the host counted.
__device__ __forceinline__ bool la_find(const LaSegments& s, int want, bool check, LaPlace* out, bool* sound) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  bool found = false, good = true;
  for (int d0 = 0; d0 < s.N; d0 += 32) {
    const int d = d0 + lane;
    int n = 0, a = 0, b = 0;
    if (d < s.N) {
      a = s.cu[d];
      b = s.cu[d + 1];
      if (a < 0 || b < a || b > s.T || (d == 0 && a != 0) || (d == s.N - 1 && b != s.T)) good = false, b = a = 0;
      n = max(1, ((b - a + LA_CH - 1) / LA_CH + s.len - 1) / s.len);
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned at = __ballot_sync(~0u, n > 0 && want >= before + sum - n && want < before + sum);
    if (at && !found) {
      const int l = __ffs(at) - 1;
      out->doc = d0 + l;
      out->index = want - before - __shfl_sync(~0u, sum - n, l);
      out->count = __shfl_sync(~0u, n, l);
      out->t0 = __shfl_sync(~0u, a, l);
      out->t1 = __shfl_sync(~0u, b, l);
      found = true;
      if (!check) break;
    }
    before += __shfl_sync(~0u, sum, 31);
  }
  *sound = __all_sync(~0u, good) && (!check || before == s.total);
  return found;
}

// waits up to about a second, whatever the error word holds from earlier calls
__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity, int* err) {
  if (mbar_drain(bar, parity)) return true;
  atomicCAS(err, 0, ST_TIMEOUT);
  return false;
}

__device__ __forceinline__ void la_tile(uint8_t* dst, const CUtensorMap* map, int head, int row, uint64_t* bar) {
  tma_load_3d(dst, map, 0, head, row, bar);
  tma_load_3d(dst + LA_TILE / 2, map, 64, head, row, bar);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

template <bool OUT, bool REV, int TERMS, bool F32>
__global__ void __launch_bounds__(LA_THREADS, 1) la_walk_kernel(const __grid_constant__ LaWalk a) {
  chain_kernel();
  extern __shared__ uint8_t la_raw[];
  uint8_t* sm = smem_align1024(la_raw);
  __shared__ uint64_t full[2], empty[2], bar_qk, bar_oi, bar_p, bar_op, bar_dz, bar_z;
  __shared__ uint32_t tmem_slot;
  __shared__ LaPlace place_s;
  __shared__ int go_s;
  __shared__ alignas(16) float pw[LA_CH + 4], back[32];   // a^d; a^(31-j): the columns of a block seen from its last
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % a.HV, want = blockIdx.x / a.HV;

  if (warp == 0) {
    LaPlace p;
    bool sound;
    const bool found = la_find(a.seg, want, blockIdx.x == 0, &p, &sound);
    if (!sound && lane == 0) atomicCAS(a.err, 0, GDN_ERR_INVALID_ARG);
    // without output: the segment that is last in the walk adds to none
    const bool go = found && sound && (OUT || (REV ? p.index > 0 : p.index + 1 < p.count));
    if (lane == 0) {
      place_s = p;
      go_s = go;
    }
  } else if (warp == 8) {
    tmem_alloc(&tmem_slot, 512);
  } else if (warp == 9 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&bar_qk, 1);
    mbar_init(&bar_oi, 1);
    mbar_init(&bar_p, LA_WORK);
    mbar_init(&bar_op, 1);
    mbar_init(&bar_dz, 1);
    mbar_init(&bar_z, LA_WORK);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const float g = [&] {
    const float x = a.decay[h];
    return x < LA_LEAST ? LA_LEAST : x;
  }();
  if (tid <= LA_CH) pw[tid] = la_power(g, (float)tid);
  if (tid < 32) back[tid] = la_power(g, (float)(31 - tid));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_slot;
  const LaPlace p = place_s;
  const int c0 = p.index * a.seg.len, chunks = (p.t1 - p.t0 + LA_CH - 1) / LA_CH;
  const int nch = go_s ? min(chunks - c0, a.seg.len) : 0;
  const bool keep = !OUT || (a.last && (REV ? p.index == 0 : p.index + 1 == p.count));   // the state at the end is wanted
  const bool from = OUT && a.init;
  // the i-th chunk of the walk: its first token, and how many
  auto first = [&](int i) { return p.t0 + (c0 + (REV ? nch - 1 - i : i)) * LA_CH; };
  auto tokens = [&](int i) { return min(LA_CH, p.t1 - first(i)); };

  if (!go_s) {
    // nothing to walk
  } else if (warp == 9) {
    // ---- loads ----
    if (lane == 0) {
      int loaded = 0;
      for (int i = 0; i < nch; ++i) {
        const int b = i & 1;
        if (i >= 2 && !la_wait(&empty[b], ((i >> 1) & 1) ^ 1, a.err)) break;
        uint8_t* st = sm + b * LA_STAGE;
        const int t = first(i);
        mbar_expect_tx(&full[b], OUT ? LA_STAGE : 2 * LA_TILE);
        la_tile(st + LA_TILE, &a.ty, h / a.gy, t, &full[b]);
        if (OUT) la_tile(st, &a.tx, h / a.gx, t, &full[b]);
        la_tile(st + 2 * LA_TILE, &a.tz, h / a.gz, t, &full[b]);
        ++loaded;
      }
      // whatever happened: what was asked for lands before the CTA ends
      for (int i = max(0, loaded - 2); i < loaded; ++i) mbar_drain(&full[i & 1], (i >> 1) & 1);
    }
  } else if (warp == 8) {
    // ---- MMAs ----
    const uint32_t zs = smem_u32(sm + LA_ZS);
    bool live = true;
    for (int i = 0; i < nch && live; ++i) {
      const int b = i & 1;
      const uint32_t x = smem_u32(sm + b * LA_STAGE), y = x + LA_TILE, z = y + LA_TILE;
      const bool add = keep || i + 1 < nch;
      if (!(live = la_wait(&full[b], (i >> 1) & 1, a.err))) break;
      if (OUT) {
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss_w(tb + LT_QK, desc_k(x, LA_CH, ks), desc_k(y, LA_CH, ks), idesc(128, 128, 0, 0), ks > 0);
        mma_commit_w(&bar_qk);
        if (!(live = la_wait(&bar_z, i & 1, a.err))) break;
        tc_fence_after();
        if (i > 0 || from) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss_w(tb + LT_OI, desc_k(x, LA_CH, ks), desc_k(zs, D, ks), idesc(128, 128, 0, 0), ks > 0);
        }
        mma_commit_w(&bar_oi);
      }
      if (!(live = la_wait(&bar_p, i & 1, a.err))) break;
      tc_fence_after();
      if (OUT) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts_w(tb + LT_OP, tb + LT_QK + (ks >> 2) * 64 + (ks & 3) * 8, desc_mn(z, LA_CH, ks), idesc(128, 128, 0, 1),
                   ks > 0);
        mma_commit_w(&bar_op);
      }
      if (add) {
        const uint32_t term[3] = {y, x, zs};
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss_w(tb + LT_DZ, desc_mn(z, LA_CH, ks), desc_mn(term[k], LA_CH, ks), idesc(128, 128, 1, 1),
                     k + ks > 0);
      }
      mma_commit_w(&bar_dz);
      mma_commit_w(&empty[b]);
    }
  } else {
    // ---- the rest: this thread's row (of tokens, or of the state) and its 64 columns ----
    const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane, col = wg * 64;
    const uint32_t tl = tb + ((uint32_t)(quad * 32) << 16);
    uint8_t* zs = sm + LA_ZS;
    float S[64];   // Z[z = row][y = col + j]
    {
      const float* src = nullptr;
      if (from) src = a.init + ((int64_t)(a.init_segments ? want : p.doc) * a.HV + h) * (D * D);
      if (!src) {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = 0.f;
      } else if (a.init_t) {
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 v = *reinterpret_cast<const float4*>(src + row * D + col + j);
          S[j] = v.x, S[j + 1] = v.y, S[j + 2] = v.z, S[j + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = src[(col + j) * D + row];
      }
    }
    auto put_state = [&](int j) {   // the columns j .. j+7 as BF16
      *reinterpret_cast<uint4*>(zs + sw_chunk(row, (col + j) >> 3, D)) =
          make_uint4(pack_bf16(S[j], S[j + 1]), pack_bf16(S[j + 2], S[j + 3]), pack_bf16(S[j + 4], S[j + 5]),
                     pack_bf16(S[j + 6], S[j + 7]));
    };
    if (OUT && nch > 0) {
#pragma unroll
      for (int j = 0; j < 64; j += 8) put_state(j);
      fence_async_smem();
      mbar_arrive(&bar_z);
    }
    bool live = true;
    for (int i = 0; i < nch && live; ++i) {
      const int b = i & 1, L = tokens(i), t = first(i);
      const bool add = keep || i + 1 < nch, state = i > 0 || from;
      uint8_t *x = sm + b * LA_STAGE, *y = x + LA_TILE, *z = y + LA_TILE;
      if (!(live = la_wait(&full[b], (i >> 1) & 1, a.err))) break;
      if (L < LA_CH) {
        // rows past the document's end are another's, or none: what they hold takes no part
        for (int k = L * 16 + tid; k < LA_CH * 16; k += LA_WORK)
          *reinterpret_cast<uint4*>(z + sw_chunk(k >> 4, k & 15, LA_CH)) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (OUT) {
        if (!(live = la_wait(&bar_qk, i & 1, a.err))) break;
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 2; ++m) {   // blocks of 32 columns: seen, not seen, or on the diagonal, as a warp's rows lie
          const int blk = wg * 2 + m;
          uint32_t w[16];
          const bool seen = REV ? blk >= quad : blk <= quad;
          if (seen) {
            float v[32];
            tmem_ld32(tl + LT_QK + blk * 32, v);
            if (blk != quad) {
              const float far = a.p_scale * (REV ? pw[blk * 32 - row] : pw[row - blk * 32 - 31]);
              const float2 f = make_float2(far, far);
              const float4* near = reinterpret_cast<const float4*>(REV ? pw : back);
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 n = near[j >> 2];
                const float2 u = mul2(make_float2(v[j], v[j + 1]), mul2(make_float2(n.x, n.y), f));
                const float2 s = mul2(make_float2(v[j + 2], v[j + 3]), mul2(make_float2(n.z, n.w), f));
                v[j] = u.x, v[j + 1] = u.y, v[j + 2] = s.x, v[j + 3] = s.y;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const int d = REV ? j - lane : lane - j;
                v[j] = d >= 0 ? v[j] * (a.p_scale * pw[max(d, 0)]) : 0.f;
              }
            }
            if (REV && L < LA_CH) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (blk * 32 + j >= L) v[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = 0u;
          }
          tmem_st8(tl + LT_QK + wg * 64 + m * 16, w);
          tmem_st8(tl + LT_QK + wg * 64 + m * 16 + 8, w + 8);
        }
        tmem_wait_st();
        tc_fence_before();
        // y and x have been read, and the state
        if (!(live = la_wait(&bar_oi, i & 1, a.err))) break;
      }
      if (add) {
#pragma unroll 2
        for (int k = tid; k < LA_CH * 16; k += LA_WORK) {
          const int c = k >> 4;
          const uint32_t at = sw_chunk(c, k & 15, LA_CH);
          const uint4 u = *reinterpret_cast<const uint4*>(y + at);
          uint32_t w[4] = {u.x, u.y, u.z, u.w}, mid[4] = {0u, 0u, 0u, 0u}, low[4] = {0u, 0u, 0u, 0u};
          if (c < L) {
            const float f = a.state_scale * pw[REV ? c + 1 : L - 1 - c];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float v0 = f * __uint_as_float(w[j] << 16), v1 = f * __uint_as_float(w[j] & 0xffff0000u);
              w[j] = pack_bf16(v0, v1);
              v0 -= __uint_as_float(w[j] << 16);
              v1 -= __uint_as_float(w[j] & 0xffff0000u);
              mid[j] = pack_bf16(v0, v1);
              if (TERMS == 3)
                low[j] = pack_bf16(v0 - __uint_as_float(mid[j] << 16), v1 - __uint_as_float(mid[j] & 0xffff0000u));
            }
          } else {
            w[0] = w[1] = w[2] = w[3] = 0u;
          }
          *reinterpret_cast<uint4*>(y + at) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(x + at) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
          if (TERMS == 3) *reinterpret_cast<uint4*>(zs + at) = make_uint4(low[0], low[1], low[2], low[3]);
        }
      }
      fence_async_smem();
      mbar_arrive(&bar_p);
      if (OUT) {
        if (!(live = la_wait(&bar_op, i & 1, a.err))) break;
        tc_fence_after();
        const float f = a.row_scale * pw[REV ? max(L - 1 - row, 0) : row + 1];
        const int64_t at = (int64_t)(t + row) * a.out_token + h * a.out_head + col;
#pragma unroll
        for (int j = 0; j < 64; j += 16) {
          float v[16];
          if (state) {
            uint32_t inter[16], intra[16];
            tmem_ld16_async(tl + LT_OI + col + j, inter);
            tmem_ld16_async(tl + LT_OP + col + j, intra);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = fmaf(f, __uint_as_float(inter[k]), __uint_as_float(intra[k]));
          } else {
            tmem_ld16(tl + LT_OP + col + j, v);
          }
          if (row < L) {
            if (F32) {
              float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + j);
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            } else {
              uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at + j);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                o[k] = make_uint4(pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]),
                                  pack_bf16(v[8 * k + 4], v[8 * k + 5]), pack_bf16(v[8 * k + 6], v[8 * k + 7]));
            }
          }
        }
      }
      if (!(live = la_wait(&bar_dz, i & 1, a.err))) break;
      tc_fence_after();
      if (add) {
        const float f = pw[L];
#pragma unroll
        for (int j = 0; j < 64; j += 16) {
          float v[16];
          tmem_ld16(tl + LT_DZ + col + j, v);
#pragma unroll
          for (int k = 0; k < 16; ++k) S[j + k] = fmaf(f, S[j + k], v[k]);
          if (OUT && i + 1 < nch) {
            put_state(j);
            put_state(j + 8);
          }
        }
      }
      tc_fence_before();
      if (OUT && i + 1 < nch) {
        fence_async_smem();
        mbar_arrive(&bar_z);
      }
    }
    if (keep && live) {
      float* dst = OUT ? a.last + ((int64_t)p.doc * a.HV + h) * (D * D) : a.sums + ((int64_t)want * a.HV + h) * (D * D);
#pragma unroll
      for (int j = 0; j < 64; ++j) dst[(col + j) * D + row] = S[j];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tb, 512);
}

// Z of each segment of a document from the sums, in the walk's order; a thread takes 4 values.
constexpr int LC_THREADS = 256, LC_PARTS = D * D / (4 * LC_THREADS), LC_AHEAD = 8;

__global__ void __launch_bounds__(LC_THREADS) la_carry_kernel(const LaCarry a) {
  chain_kernel();
  const int part = blockIdx.x % LC_PARTS, h = blockIdx.x / LC_PARTS % a.HV, doc = blockIdx.x / LC_PARTS / a.HV;
  // the segments before the document
  __shared__ int before_s, bad_s;
  if (threadIdx.x < 32) {
    int before = 0;
    bool bad = false;
    for (int d = threadIdx.x; d < doc; d += 32) {
      const int n = a.seg.cu[d + 1] - a.seg.cu[d];
      bad |= n < 0 || n > a.seg.T;
      before += max(1, ((max(n, 0) + LA_CH - 1) / LA_CH + a.seg.len - 1) / a.seg.len);
    }
    before = __reduce_add_sync(~0u, before);
    bad = __any_sync(~0u, bad);
    if (threadIdx.x == 0) before_s = before, bad_s = bad;
  }
  __syncthreads();
  const int n = a.seg.cu[doc + 1] - a.seg.cu[doc];
  const int chunks = (n + LA_CH - 1) / LA_CH, count = max(1, (chunks + a.seg.len - 1) / a.seg.len);
  if (bad_s || n < 0 || n > a.seg.T || before_s + count > a.seg.total) {
    if (threadIdx.x == 0) atomicCAS(a.err, 0, GDN_ERR_INVALID_ARG);
    return;
  }
  float g = a.decay[h];
  if (g < LA_LEAST) g = LA_LEAST;
  const int e = (part * LC_THREADS + threadIdx.x) * 4, y = e / D, z = e % D;
  float Z[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.init) {
    const float* s = a.init + ((int64_t)doc * a.HV + h) * (D * D);
#pragma unroll
    for (int k = 0; k < 4; ++k) Z[k] = a.init_t ? s[(z + k) * D + y] : s[e + k];
  }
  const float whole = la_power(g, (float)(a.seg.len * LA_CH));
  const float rest = la_power(g, (float)(n - (count - 1) * a.seg.len * LA_CH));   // of the last segment
  const int64_t pitch = (int64_t)a.HV * (D * D);
  float* at = a.sums + ((int64_t)before_s * a.HV + h) * (D * D) + e;
  for (int i0 = 0; i0 < count; i0 += LC_AHEAD) {
    float4 add[LC_AHEAD];
#pragma unroll
    for (int k = 0; k < LC_AHEAD; ++k) {
      const int i = i0 + k, s = a.reverse ? count - 1 - i : i;
      if (i + 1 < count) add[k] = *reinterpret_cast<const float4*>(at + s * pitch);
    }
#pragma unroll
    for (int k = 0; k < LC_AHEAD; ++k) {
      const int i = i0 + k, s = a.reverse ? count - 1 - i : i;
      if (i < count) {
        *reinterpret_cast<float4*>(at + s * pitch) = make_float4(Z[0], Z[1], Z[2], Z[3]);
        const float f = s == count - 1 ? rest : whole;
        if (i + 1 < count) {
          Z[0] = fmaf(f, Z[0], add[k].x);
          Z[1] = fmaf(f, Z[1], add[k].y);
          Z[2] = fmaf(f, Z[2], add[k].z);
          Z[3] = fmaf(f, Z[3], add[k].w);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(256) la_reduce_kernel(const float* part, __nv_bfloat16* out, int64_t items, int H, int G,
                                                        int64_t out_token) {
  chain_kernel();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < items; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t th = i >> 4;   // token, head
    const float4* p = reinterpret_cast<const float4*>(part + th * G * D) + (i & 15) * 2;
    float4 u = p[0], v = p[1];
    for (int k = 1; k < G; ++k) {
      const float4 s = p[k * 32], w = p[k * 32 + 1];
      u.x += s.x, u.y += s.y, u.z += s.z, u.w += s.w;
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    *reinterpret_cast<uint4*>(out + th / H * out_token + th % H * D + (i & 15) * 8) =
        make_uint4(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w), pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
}

template <bool OUT, bool REV, int TERMS, bool F32> static cudaError_t launch_walk(const LaWalk& a, cudaStream_t s) {
  const auto kernel = la_walk_kernel<OUT, REV, TERMS, F32>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LA_SMEM);
  if (e != cudaSuccess) return e;
  return launch_chained(kernel, dim3((unsigned)a.seg.total * a.HV), dim3(LA_THREADS), LA_SMEM, s, a);
}

cudaError_t launch_la_walk(const LaWalk& a, bool reverse, int terms, bool f32, cudaStream_t s) {
  if (reverse) {
    if (f32) return launch_walk<true, true, 2, true>(a, s);
    return terms == 3 ? launch_walk<true, true, 3, false>(a, s) : launch_walk<true, true, 2, false>(a, s);
  }
  if (f32) return launch_walk<true, false, 2, true>(a, s);
  return terms == 3 ? launch_walk<true, false, 3, false>(a, s) : launch_walk<true, false, 2, false>(a, s);
}

cudaError_t launch_la_sums(const LaWalk& a, bool reverse, cudaStream_t s) {
  return reverse ? launch_walk<false, true, 3, false>(a, s) : launch_walk<false, false, 3, false>(a, s);
}

cudaError_t launch_la_carry(const LaCarry& a, cudaStream_t s) {
  return launch_chained(la_carry_kernel, dim3((unsigned)(a.seg.N * a.HV * LC_PARTS)), dim3(LC_THREADS), 0, s, a);
}

cudaError_t launch_la_reduce(const float* part, void* out, int64_t T, int H, int G, int64_t out_token, cudaStream_t s) {
  const int64_t items = T * H * 16;
  const int64_t blocks = (items + 255) / 256;
  return launch_chained(la_reduce_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, part,
                        static_cast<__nv_bfloat16*>(out), items, H, G, out_token);
}

}  // namespace gdn
