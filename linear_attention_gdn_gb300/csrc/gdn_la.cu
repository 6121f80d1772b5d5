// gdn_la.cu -- linear attention with a fixed decay a per head, in chunks of L <= 128 tokens.
//
// Every result of the forward and the backward is one walk over the chunks of a document, with rows x, y, z of 128 values:
//   out_r = sum_{c seen by r} a^|r-c| (x_r . y_c) z_c + a^(tokens between) Z^T x_r,     Z <- a^L Z + sum_c a^.. y_c z_c^T
//   forward  o : x, y, z = q, k, v;     dq : dO, v, k     (r sees c <= r; Z is the state before the chunk)
//   reverse  dv: x, y, z = k, q, dO;    dk : v, dO, q     (r sees c >= r; Z is the gradient behind the chunk)
//
// A CTA walks one segment of a document for one value head.  Per chunk, on the tensor cores:
//   QK[r][c] = x_r . y_c;  O = x Z;  dZ[y][z] = (decayed y)^T z;  P = decayed, masked QK;  O = a^.. O + P z
// P and the decayed y go to TMEM as left operands, so that shared memory, which all operands pass, is read least.  The state
// is FP32 in registers (thread: one row y, 64 columns z), rounded to BF16 once for the product with x.  The decayed y is given
// to the product as a sum of BF16 terms, so that the state keeps FP32's exactness: two terms (2^-17) where only BF16 results
// come of it, by the packed BF16 multiply-add, whose rounding the next one recovers (3 instructions a pair of values); three, the
// whole FP32 product 8 bits at a time, where the state itself is handed out.
// Three sets of warps work side by side: one makes P, scales O and writes it out, one makes the decayed y, a quarter of a
// chunk at a time in a ring, one carries the state on; so the tensor cores have dZ to do while P is made.
// Documents whose chains are too few or too long are cut into segments: la_walk without output first sums what each adds,
// la_carry_kernel turns the sums into the states they start from.
//
// Heads of a group share q and k: dq and dk are sums over them.  Each head is a CTA; the first stores its part of a chunk, the
// next add theirs by the memory system, the last loads the sum before it and writes the result, each when the one before has
// (3 documents of 8,192 tokens, 48 heads on 16: a walk with sums 252 us, without 167).
//
// What bounds it: a chunk is 12.6 MFLOP of products (6 of 128^3; dZ two or three times) and 128 KB to and from memory, and
// takes a CTA 2.5 to 2.9 us (3 documents of 8,192 tokens, 48 heads of their own: 185 us, 6.5 TB/s, 96% of a plain copy's rate;
// of 32,768 tokens 699 us, 6.9 TB/s).  By the counters the tensor cores work half of the time and the warps issue 56%: it is the
// chain from QK to the output of one chunk, of which the next chunk's can overlap all but P.  Where heads share q and k, memory
// has less to do and the chunk's time stays (12 prompts of 30,054 tokens in all, 48 heads on 16: 266 us, 59% of the copy rate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_la.cuh"
#include "gdn_launch.cuh"

namespace gdn {

constexpr int LA_SET = 256;                   // threads of each of the three sets: two warpgroups
constexpr int LA_THREADS = 3 * LA_SET + 128;  // and a warp each for the loads, two streams of MMAs, the sums' output
constexpr int LA_MMA = 3 * LA_SET / 32, LA_LOAD = LA_MMA + 1, LA_DZ = LA_MMA + 2, LA_SUM = LA_MMA + 3;   // those warps
// Registers a thread, of the 72 that the CTA is launched with: 256 x (80 + 56 + 96) + 128 x 40 = 896 x 72
constexpr int LA_REG_OUT = 80, LA_REG_Y = 56, LA_REG_STATE = 96, LA_REG_CTRL = 40;
constexpr int LA_TILE = LA_CH * D * 2;       // 32 KB
constexpr int LA_STAGE = 3 * LA_TILE;        // y, x, z; z then has the output on its way out (FP32: x and z)
constexpr int LA_Y = 0, LA_X = LA_TILE, LA_Z = 2 * LA_TILE;
constexpr int LA_ZS = 2 * LA_STAGE;          // the state as BF16 [y][z]
constexpr int LA_SMEM = LA_ZS + LA_TILE + 1024;
// TMEM columns: QK, each 16 of them then P in their first 8; O; dZ; the ring of decayed y
constexpr int LT_QK = 0, LT_O = 128, LT_DZ = 256, LT_Y = 384;
constexpr int LA_Q = 32;                     // tokens of a quarter: 16 columns a term
constexpr int LA_SHORT = 64;                 // tokens of a chunk whose P has two terms, in as many products as a whole one's
constexpr float LA_COLUMNS = -0.7f;   // (64 times it: 2^-65, which leaves P z as much of FP32's range)
constexpr float LA_LEAST = -1e4f;   // log decays below it: nothing is left of it either, and no product is NaN

// a^n: the product's rounding error is put back, so that far powers are as exact as near ones
__device__ __forceinline__ float la_power(float g, float n) {
  const float p = g * n, e = expf(p);
  return fmaf(e, fmaf(g, n, -p), e);
}

// from L2 in kernels that may follow another without waiting
template <bool L2, typename T> __device__ __forceinline__ T la_load(const T* p) { return L2 ? __ldcg(p) : *p; }

struct LaPlace {
  int doc, index, count;   // segment `index` of the document's `count`
  int segment;             // its number among all
  int t0, t1;              // the document's tokens
};

// The segment of place `want` by one warp; false if there is none, if the documents up to it are not in order, or if its
// document's segments do not all have numbers below the host's count (which is all that there is memory for; a place below it
// alone says nothing of its segment's number where places go by length).  If `check`, the whole list is walked, and *sound
// tells whether it is in order and the host's.  Up to 32 documents give their segments by falling length,
// so that no long one begins when the others end (12 prompts of up to 4,096 tokens).
template <bool L2> __device__ __forceinline__ bool la_find(const LaSegments& s, int want, bool check, LaPlace* out, bool* sound) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  bool found = false, good = true, there = false;
  uint64_t bounds = 0;   // of this lane's documents
#pragma unroll 1
  for (int d0 = 0; d0 < s.N; d0 += 32) {
    int d = d0 + lane;
    int n = 0, a = 0, b = 0;
    if (d < s.N) {
      a = la_load<L2>(s.cu + d);
      b = la_load<L2>(s.cu + d + 1);
      if (check) bounds += la_bound(d, b);
      if (a < 0 || b < a || b > s.T || (d == 0 && a != 0) || (d == s.N - 1 && b != s.T)) good = false, b = a = 0;
      n = max(1, ((b - a + LA_CH - 1) / LA_CH + s.len - 1) / s.len);
    }
    auto sums = [&](int x) {   // inclusive, over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      return x;
    };
    int first = before + sums(n) - n, place = first;   // of the document's segments: their number, their place
    if (s.N > 1 && s.N <= 32) {
      const int key = d < s.N ? min(b - a, s.len * LA_CH) : -1;
      int rank = 0, from = 0;
#pragma unroll 4
      for (int i = 0; i < s.N; ++i) {
        const int other = __shfl_sync(~0u, key, i);
        rank += other > key || (other == key && i < lane);
      }
#pragma unroll 4
      for (int i = 0; i < s.N; ++i)
        if (__shfl_sync(~0u, rank, i) == lane) from = i;
      d = from;
      n = __shfl_sync(~0u, n, from);
      if (lane >= s.N) n = 0;
      a = __shfl_sync(~0u, a, from);
      b = __shfl_sync(~0u, b, from);
      first = __shfl_sync(~0u, first, from);
      place = sums(n) - n;
    }
    good = __all_sync(~0u, good);
    const unsigned at = __ballot_sync(~0u, n > 0 && want >= place && want < place + n);
    if (at && !there) {
      const int l = __ffs(at) - 1;
      out->doc = __shfl_sync(~0u, d, l);
      out->index = want - __shfl_sync(~0u, place, l);
      out->segment = __shfl_sync(~0u, first, l) + out->index;
      out->count = __shfl_sync(~0u, n, l);
      out->t0 = __shfl_sync(~0u, a, l);
      out->t1 = __shfl_sync(~0u, b, l);
      there = true;
      found = good && out->segment - out->index + out->count <= s.total;
      if (!check) break;
    }
    before += __shfl_sync(~0u, sums(n), 31);
  }
  if (check) {
#pragma unroll
    for (int o = 16; o; o >>= 1) bounds += __shfl_xor_sync(~0u, bounds, o);
    good = good && bounds == s.bounds;
  }
  *sound = good;
  return found;
}

// Waits, but not for ever: 2^18 tries of up to 4 us each, about a second; false if they run out.  Small on purpose, as are the
// loops below: the kernel's speed is lost as soon as its code leaves the instruction cache (with the waits and loops unrolled it
// had 196 KB, and a chunk took 12,000 cycles; now 4,700).
__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
#pragma unroll 1
  for (uint32_t i = 0; i < 1u << 18; ++i) {
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) break;
  }
  return done;
}

// A warp's arrival: one for its 32 threads (counted one by one they queue at the barrier's word: 256 take 500 cycles).
__device__ __forceinline__ void la_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A count in memory that another CTA raises (2^20 tries: about a second, too).
__device__ __forceinline__ bool la_wait_count(const int* count, int least) {
#pragma unroll 1
  for (uint32_t i = 0; i < 1u << 20; ++i) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
    if (v >= least) return true;
    __nanosleep(40);
  }
  return false;
}
// a tile of a sum to memory, added to what is there, and back
__device__ __forceinline__ void la_bulk_store(float* dst, const void* ssrc, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(ssrc)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void la_bulk_add(float* dst, const void* ssrc, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(ssrc)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void la_bulk_load(void* sdst, const float* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(sdst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// barrier over one set that also tells whether all of it is well
template <int ID, int N> __device__ __forceinline__ bool la_set_well(bool v) {
  asm volatile("" ::: "memory");
  v = bar_and(ID, N, v);
  asm volatile("" ::: "memory");
  return v;
}

__device__ __forceinline__ void la_tile(uint8_t* dst, const CUtensorMap* map, int head, int row, uint64_t* bar) {
  tma_load_3d(dst, map, 0, head, row, bar);
  tma_load_3d(dst + LA_TILE / 2, map, 64, head, row, bar);
}

__device__ __forceinline__ void la_prefetch(const CUtensorMap* map, int head, int row) {
  tma_prefetch_3d(map, 0, head, row);
  tma_prefetch_3d(map, 64, head, row);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// pairs of BF16 values: products and sums rounded once
__device__ __forceinline__ uint32_t bf_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// a pair of FP32 values as two pairs of BF16 whose sums they are (to 2^-17)
__device__ __forceinline__ void la_parts(float2 v, uint32_t (&part)[2]) {
  part[0] = pack_bf16(v.x, v.y);
  part[1] = pack_bf16(v.x - __uint_as_float(part[0] << 16), v.y - __uint_as_float(part[0] & 0xffff0000u));
}
// BF16 by cutting off: the upper halves of two values, and what is left of them below
__device__ __forceinline__ uint32_t uppers(float2 x) {
  return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
__device__ __forceinline__ float2 below(float2 x) {
  const float2 top = make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u), __uint_as_float(__float_as_uint(x.y) & 0xffff0000u));
  return __ffma2_rn(top, make_float2(-1.f, -1.f), x);
}

// 16 lanes x 8 columns: register 2 m + i of a lane goes to the TMEM lane (lane / 4) + 8 i, column 4 m + lane % 4
__device__ __forceinline__ void tmem_st_16lanes(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]));
}

// byte offset of the 16-byte piece c16 (of 32) of row r in an FP32 [128][128] tile, swizzled as the BF16 ones
__device__ __forceinline__ uint32_t la_f32(int r, int c16) {
  return (uint32_t)((c16 >> 3) * (LA_CH * 128) + r * 128 + (((c16 & 7) ^ (r & 7)) << 4));
}

// the same where a warp's 32 rows lie side by side, and the first 32 of each 64 columns in the first half
__device__ __forceinline__ uint32_t la_part(int r, int c16) {
  return (uint32_t)((((c16 & 8) << 1) + ((c16 & 16) >> 1) + (c16 & 7)) * LA_CH + r) * 16;
}

template <bool OUT, bool REV, int TERMS, bool SUM>
__global__ void __launch_bounds__(LA_THREADS, 1) la_walk_kernel(const __grid_constant__ LaWalk a) {
  constexpr bool LEADS = OUT && REV && !SUM, FOLLOWS = OUT && TERMS == 2;   // (which may)
  if (!LEADS || !a.leads) dependents_may_launch();
  constexpr int SLOTS = OUT ? 128 / (16 * TERMS) : 4;   // of the ring
  // without output there is room for the ring of a whole chunk and for a second dZ, made while the first is read
  constexpr int T_Y = OUT ? LT_Y : 256;
  auto t_dz = [](int i) { return OUT ? LT_DZ : (i & 1) * 128; };
  extern __shared__ uint8_t la_raw[];
  uint8_t* sm = smem_align1024(la_raw);
  // a tile is asked for again as soon as it has been used: y by QK and the decayed y, x by O, z at the end of its chunk
  __shared__ uint64_t full_y[2], full_x[2], full_z[2], empty_y[2], empty_x[2], empty_z[2], y_full[SLOTS], y_empty[4];
  // (by the chunk's parity: dZ may be a chunk ahead of those that wait for it, and these do not all wait in every chunk)
  __shared__ uint64_t bar_dz[2], dz_read[2], bar_oi[2];
  // SUM: this head's part is there, may be loaded over; the sum of the heads before it, by halves
  __shared__ uint64_t part_full[2], part_empty[2], part_in[2][2];
  __shared__ uint64_t bar_qk, bar_p, bar_op, bar_o, bar_z, bar_init;
  __shared__ uint32_t tmem_slot;
  __shared__ LaPlace place_s;
  __shared__ int go_s, h_s;
  // a^d; P's factors where they go by columns alone (the first half's); the decayed y's factors in a whole chunk
  __shared__ alignas(16) float pw[LA_CH + 4], wcol[LA_CH / 2];
  __shared__ uint32_t fy[2][LA_CH / 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // what touches no memory, while the kernel before ends
  if (warp == LA_MMA) {
    tmem_alloc(&tmem_slot, 512);
  } else if (warp == LA_LOAD && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full_y[i], 1);
      mbar_init(&full_x[i], 1);
      mbar_init(&full_z[i], 1);
      mbar_init(&bar_dz[i], 1);
      mbar_init(&dz_read[i], LA_SET / 32);
      mbar_init(&bar_oi[i], 1);
      mbar_init(&empty_y[i], OUT ? LA_SET / 32 + 1 : 2 * LA_SET / 32);
      mbar_init(&empty_x[i], 1);
      mbar_init(&empty_z[i], OUT ? 3 : 1);
      mbar_init(&part_in[0][i], 1);
      mbar_init(&part_in[1][i], 1);
      mbar_init(&part_full[i], 1);
      mbar_init(&part_empty[i], 1);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&y_full[i], 4);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&y_empty[i], 1);
    mbar_init(&bar_qk, 1);
    mbar_init(&bar_p, LA_SET / 32);
    mbar_init(&bar_op, 1);
    mbar_init(&bar_o, LA_SET / 32);
    mbar_init(&bar_z, LA_SET / 32);
    mbar_init(&bar_init, LA_SET / 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == LA_DZ && lane == 0) {
    const CUtensorMap* maps[4] = {&a.tx, &a.ty, &a.tz, &a.to};
#pragma unroll
    for (int i = OUT ? 0 : 1; i < (OUT ? 4 : 3); ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(maps[i]) : "memory");
  }
  if (!FOLLOWS || !a.follows) previous_kernel_done();   // (else the kernels before it, but one, have ended; what is read comes from L2)
  if (LEADS && a.leads) dependents_may_launch();
  // SUM: in the order in which CTAs begin, so that what a head waits for has begun before it, whatever runs side by side
  int number = blockIdx.x;
  if (SUM) {
    if (tid == 0) h_s = atomicAdd(a.ticket, 1);
    __syncthreads();
    number = h_s;
  }
  const int h = number % a.HV, want = number / a.HV;
  const int head = SUM ? h / a.group : h, rank = SUM ? h % a.group : 0;
  const bool ends = !SUM || rank + 1 == a.group;   // (the last head of a group has the sum)
  if (warp == 0) {
    LaPlace p;
    bool sound;
    const bool found = la_find<FOLLOWS>(a.seg, want, number == 0, &p, &sound);   // (all heads find the same)
    if (!sound && lane == 0) atomicCAS(a.err, 0, GDN_ERR_INVALID_ARG);
    // without output: the segment that is last in the walk adds to none; without states of segments: a document has one, or
    // it is not the host's
    const bool go = found && (OUT ? a.init_segments || p.count == 1 : REV ? p.index > 0 : p.index + 1 < p.count);
    if (lane == 0) {
      place_s = p;
      go_s = go;
    }
  }
  const float g = [&] {
    const float x = la_load<FOLLOWS>(a.decay + h);
    return x < LA_LEAST ? LA_LEAST : x;
  }();
  // Where a^-64 is no more than 2^65, a^(r-c) is a^(63-c) in P and a^(r-63) on O at the end, and the state's part comes by
  // a state that is held as a^64 of it, without a pass over O between (12 prompts, all decays -0.69: 250 us, -0.71: 283).
  const bool columns = OUT && g >= LA_COLUMNS && a.row_scale != 0.f;
  const float held = columns ? la_power(g, 64.f) : 1.f;
  if (tid <= LA_CH) pw[tid] = la_power(g, (float)tid);
  if (tid >= 256 && tid < 256 + LA_CH / 2 && columns) {
    const int c = tid - 256;
    wcol[c] = a.p_scale / a.row_scale * la_power(g, (float)(REV ? c - 63 : 63 - c));
  }
  if (tid >= 384 && tid < 384 + LA_CH / 2) {
    const int c = (tid - 384) * 2;
    const float2 f = make_float2(a.state_scale * held * la_power(g, (float)(REV ? c + 1 : LA_CH - 1 - c)),
                                 a.state_scale * held * la_power(g, (float)(REV ? c + 2 : LA_CH - 2 - c)));
    uint32_t part[2] = {__float_as_uint(f.x), __float_as_uint(f.y)};
    if (TERMS == 2) la_parts(f, part);
    fy[0][c >> 1] = part[0];
    fy[1][c >> 1] = part[1];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_slot;
  const LaPlace p = place_s;
  const int c0 = p.index * a.seg.len, chunks = (p.t1 - p.t0 + LA_CH - 1) / LA_CH;
  const int nch = go_s ? min(chunks - c0, a.seg.len) : 0;
  const bool keep = !OUT || (a.last && (REV ? p.index == 0 : p.index + 1 == p.count));   // the state at the end is wanted
  const bool from = OUT && a.init;
  const int adds = keep ? nch : max(nch - 1, 0);   // chunks that add to the state
  bool live = true;   // no wait has run out
  const bool staged = from && !a.init_t;   // the first state comes by way of the second stage
  // the i-th chunk of the walk: its first token, and how many
  auto first = [&](int i) { return p.t0 + (c0 + (REV ? nch - 1 - i : i)) * LA_CH; };
  auto tokens = [&](int i) { return min(LA_CH, p.t1 - first(i)); };

  // ---- the decayed y, by one warpgroup the quarters q0, q0 + qs, ..; a warp 32 columns of y ----
  auto make_y = [&](int q0, int qs) {
    const int quad = warp & 3;
    const uint32_t tl = tb + ((uint32_t)(quad * 32) << 16);
    // Quarter q of chunk i, in terms.  A transposing load gives a lane the tokens 2 (lane % 4) and the next of the column
    // lane / 4 of each 8 x 8 block, which is also how a store of 16 TMEM lanes takes them.
    auto quarter = [&](int i, int q) {
      const int n = i * 4 + q, slot = n % SLOTS, L = tokens(i);
      const uint32_t to = tl + T_Y + slot * TERMS * 16;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {   // 16 tokens
        const int t0 = q * LA_Q + half * 16, pair = (lane & 3) * 2;
        uint32_t y[8];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int c8 = quad * 4 + m * 2 + ((lane >> 3) & 1), r = t0 + (lane >> 4) * 8 + (lane & 7);
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(y[4 * m]), "=r"(y[4 * m + 1]), "=r"(y[4 * m + 2]), "=r"(y[4 * m + 3])
                       : "r"(smem_u32(sm + (i & 1) * LA_STAGE + LA_Y) + sw_chunk(r, c8, LA_CH))
                       : "memory");
        }
        // The decays of this lane's tokens in the first and the last 8 as two BF16 parts each, or, for a state that is
        // handed out, in FP32; and the products in BF16 parts: y f1 and what its rounding left (exact: 16 bits) with y f2; or
        // the FP32 product's three times 8 bits.
        uint32_t w[TERMS][8];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int c = t0 + m * 8 + pair;
          float2 f;
          uint32_t part[2];
          if (L == LA_CH) {
            if (TERMS == 2) part[0] = fy[0][c >> 1], part[1] = fy[1][c >> 1];
            else f = make_float2(__uint_as_float(fy[0][c >> 1]), __uint_as_float(fy[1][c >> 1]));
          } else {
            f.x = c < L ? a.state_scale * held * pw[REV ? c + 1 : L - 1 - c] : 0.f;
            f.y = c + 1 < L ? a.state_scale * held * pw[REV ? c + 2 : L - 2 - c] : 0.f;
            la_parts(f, part);
            // what the rows past the end hold takes no part
            const uint32_t mask = (c < L ? 0xffffu : 0u) | (c + 1 < L ? 0xffff0000u : 0u);
            y[2 * m] &= mask, y[2 * m + 1] &= mask, y[4 + 2 * m] &= mask, y[5 + 2 * m] &= mask;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 2 * m + (e & 1) + (e >> 1) * 4;
            if (TERMS == 2) {
              w[0][k] = bf_mul(y[k], part[0]);
              w[1][k] = bf_fma(y[k], part[1], bf_fma(y[k], part[0], w[0][k] ^ 0x80008000u));
            } else {
              float2 v = mul2(f, make_float2(__uint_as_float(y[k] << 16), __uint_as_float(y[k] & 0xffff0000u)));
#pragma unroll
              for (int n = 0; n < TERMS; ++n) {
                w[n][k] = uppers(v);
                v = below(v);
              }
            }
          }
        }
        if (half == 0) {
          // (of the quarter that had the slot before; so that each warpgroup sees every phase of the one barrier it waits for)
          if (n >= SLOTS && !(live = la_wait(&y_empty[(q - SLOTS) & 3], ((n - SLOTS) >> 2) & 1))) return;
          tc_fence_after();
        }
#pragma unroll
        for (int e = 0; e < TERMS; ++e) {
          tmem_st_16lanes(to + e * 16 + half * 8, w[e]);
          tmem_st_16lanes(to + e * 16 + half * 8 + (16u << 16), w[e] + 4);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      la_arrive(&y_full[slot]);
    };
    const int steps = go_s ? adds : 0;
#pragma unroll 1
    for (int i = 0; i < steps && live; ++i) {
      if (!(live = la_wait(&full_y[i & 1], (i >> 1) & 1))) break;
      const int L = tokens(i);
#pragma unroll 1
      for (int q = q0; q < 4 && live; q += qs) {
        if (L < LA_CH) {   // z of the rows past the end, as far as this quarter's products read them
          if (!(live = la_wait(&full_z[i & 1], (i >> 1) & 1))) break;
          uint8_t* z = sm + (i & 1) * LA_STAGE + LA_Z;
#pragma unroll 1
          for (int k = max(L, q * LA_Q) * 16 + (tid & 127); k < (q + 1) * LA_Q * 16; k += 128)
            *reinterpret_cast<uint4*>(z + sw_chunk(k >> 4, k & 15, LA_CH)) = make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();
        }
        quarter(i, q);
      }
      la_arrive(&empty_y[i & 1]);
    }
  };

  if (warp >= LA_MMA) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LA_REG_CTRL));
    if (warp == LA_LOAD && lane == 0 && go_s) {
      // ---- loads ----
      int ny = 0, nx = 0, nz = 0;   // asked for
#pragma unroll 1
      for (int i = 0; i < nch && live; ++i) {
        const int b = i & 1, t = first(i);
        const uint32_t free = ((i >> 1) & 1) ^ 1;
        uint8_t* st = sm + b * LA_STAGE;
        if (i == 1 && staged && !(live = la_wait(&bar_init, 0))) break;
        if (i >= 2 && !(live = la_wait(&empty_y[b], free))) break;
        if (SUM && i >= 2 && !(live = la_wait(&part_empty[b], free))) break;
        mbar_expect_tx(&full_y[b], LA_TILE);
        la_tile(st + LA_Y, &a.ty, h / a.gy, t, &full_y[b]);
        ++ny;
        if (OUT) {
          if (i >= 2 && !(live = la_wait(&empty_x[b], free))) break;
          mbar_expect_tx(&full_x[b], LA_TILE);
          la_tile(st + LA_X, &a.tx, h / a.gx, t, &full_x[b]);
          ++nx;
        }
        if (i >= 2 && !(live = la_wait(&empty_z[b], free))) break;
        mbar_expect_tx(&full_z[b], LA_TILE);
        la_tile(st + LA_Z, &a.tz, h / a.gz, t, &full_z[b]);
        ++nz;
        if (i + 2 < nch) {   // until their tiles are free, the next rows come as far as L2
          const int ahead = first(i + 2);
          la_prefetch(&a.ty, h / a.gy, ahead);
          if (OUT) la_prefetch(&a.tx, h / a.gx, ahead);
          la_prefetch(&a.tz, h / a.gz, ahead);
        }
      }
      // whatever happened: what was asked for lands before the CTA ends
#pragma unroll 1
      for (int i = max(0, ny - 2); i < ny; ++i) mbar_drain(&full_y[i & 1], (i >> 1) & 1);
#pragma unroll 1
      for (int i = max(0, nx - 2); i < nx; ++i) mbar_drain(&full_x[i & 1], (i >> 1) & 1);
#pragma unroll 1
      for (int i = max(0, nz - 2); i < nz; ++i) mbar_drain(&full_z[i & 1], (i >> 1) & 1);
    }
    // ---- the products, in two streams that wait for different things: QK, x Z and P z here ----
    if (OUT && warp == LA_MMA && go_s) {
      const uint32_t zs = smem_u32(sm + LA_ZS);
#pragma unroll 1
      for (int i = 0; i < nch && live; ++i) {
        const int b = i & 1;
        const uint32_t par = (i >> 1) & 1, st = smem_u32(sm + b * LA_STAGE), x = st + LA_X, z = st + LA_Z;
        if (!(live = la_wait(&full_y[b], par) && la_wait(&full_x[b], par))) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss_w(tb + LT_QK, desc_k(x, LA_CH, ks), desc_k(st + LA_Y, LA_CH, ks), idesc(128, 128, 0, 0), ks > 0);
        mma_commit_w(&bar_qk);
        mma_commit_w(&empty_y[b]);
        if (!(live = la_wait(&bar_z, i & 1))) break;
        if (i > 0 && !(live = la_wait(&bar_o, (i - 1) & 1))) break;
        tc_fence_after();
        if (i > 0 || from) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss_w(tb + LT_O, desc_k(x, LA_CH, ks), desc_mn(zs, D, ks), idesc(128, 128, 0, 1), ks > 0);
        }
        mma_commit_w(&bar_oi[b]);
        mma_commit_w(&empty_x[b]);
        // (P's second terms meet the same rows of z as the first)
        const uint32_t upper = z + (tokens(i) <= LA_SHORT ? 0 : LA_SHORT * 128);
        if (!(live = la_wait(&bar_p, i & 1) && la_wait(&full_z[b], par))) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts_w(tb + LT_O, tb + LT_QK + ks * 16, desc_mn(ks < 4 ? z : upper, LA_CH, ks & 3), idesc(128, 128, 0, 1),
                   ks > 0 || i > 0 || from);
        mma_commit_w(&bar_op);
        mma_commit_w(&empty_z[b]);
      }
    }
    // ---- SUM: the parts go out from where y and x were, each head's added to those before it, by the memory system but in the
    // heads' order; the last head has the sum before it come in there ----
    if (SUM && warp == LA_SUM && lane == 0 && go_s) {
      // the chunk's number (no two documents' chunks have the same), whose tile, and how many heads are in it
      auto place = [&](int i) { return ((int64_t)p.t0 / LA_CH + p.doc + (first(i) - p.t0) / LA_CH) * (a.HV / a.group) + head; };
      int in = 0;   // halves asked for
#pragma unroll 1
      for (int i = 0; i < nch && live; ++i) {
        const int b = i & 1;
        const uint32_t par = (i >> 1) & 1;
        uint8_t* tile = sm + b * LA_STAGE + LA_Y;
        float* to = a.sums + place(i) * (LA_CH * D);
        int* count = a.counts + place(i);
        if (ends) {
          if (!(live = la_wait_count(count, rank) && (i >= adds || la_wait(&empty_y[b], par)))) break;
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            if ((k || i >= adds) && !(live = la_wait(&empty_x[b], par))) break;
            asm volatile("fence.proxy.async;" ::: "memory");
            mbar_expect_tx(&part_in[k][b], LA_TILE);
            la_bulk_load(tile + k * LA_TILE, to + k * (LA_CH * D / 2), LA_TILE, &part_in[k][b]);
            ++in;
          }
          continue;
        }
        if (!(live = la_wait(&part_full[b], par) && (rank == 0 || la_wait_count(count, rank)))) break;
        asm volatile("fence.proxy.async.global;" ::: "memory");
        if (rank == 0) la_bulk_store(to, tile, 2 * LA_TILE);
        else la_bulk_add(to, tile, 2 * LA_TILE);
        bulk_commit();
        bulk_wait_read();
        mbar_arrive(&part_empty[b]);
        bulk_wait_all();
        asm volatile("fence.proxy.async.global;" ::: "memory");
        asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(count), "r"(rank + 1) : "memory");
      }
#pragma unroll 1
      for (int i = max(0, in - 4); i < in; ++i) mbar_drain(&part_in[i & 1][(i >> 1) & 1], (i >> 2) & 1);
    }
    // ---- and dZ here ----
    if (warp == LA_DZ && go_s) {
#pragma unroll 1
      for (int n = 0; n < 4 * adds && live; ++n) {
        const int i = n >> 2, q = n & 3, slot = n % SLOTS;
        const uint32_t z = smem_u32(sm + (i & 1) * LA_STAGE + LA_Z);
        if (q == 0) {
          const int last = OUT ? i - 1 : i - 2;   // chunk whose dZ was where this one's goes
          if (last >= 0 && !(live = la_wait(&dz_read[last & 1], (last >> 1) & 1))) break;
          if (!(live = la_wait(&full_z[i & 1], (i >> 1) & 1))) break;
        }
        if (!(live = la_wait(&y_full[slot], (n / SLOTS) & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            mma_ts_w(tb + t_dz(i), tb + T_Y + (slot * TERMS + k) * 16 + ks * 8, desc_mn(z, LA_CH, q * 2 + ks),
                     idesc(128, 128, 0, 1), q + k + ks > 0);
        mma_commit_w(&y_empty[q]);
        if (q == 3) {
          mma_commit_w(&bar_dz[i & 1]);
          mma_commit_w(&empty_z[i & 1]);
        }
      }
    }
  } else if (warp < LA_SET / 32) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LA_REG_OUT));
    // ---- P and O: this thread's row of tokens and its 64 columns (without output: half of the quarters, too) ----
    if (!OUT) {
      make_y((tid >> 7) & 1, 4);
    } else if (go_s) {
      const int wg = warp >> 2, quad = warp & 3, row = quad * 32 + lane, col = wg * 64;
      const uint32_t tl = tb + ((uint32_t)(quad * 32) << 16);
      const float half = columns ? la_power(g, REV ? 64.f : -64.f) : 1.f;
      // O's factor: of this row in a whole chunk, as P goes by columns; else of the state's part
      const float whole = columns ? a.row_scale * la_power(g, (float)(REV ? 63 - row : row - 63)) : 0.f;
      const float back = columns ? a.row_scale * la_power(g, -64.f) : a.row_scale;
      auto sent = [&](int i) {   // chunk i's output has left its tiles
        bulk_wait_read();
        mbar_arrive(&empty_z[i & 1]);
      };
#pragma unroll 1
      for (int i = 0; i < nch && live; ++i) {
        const int b = i & 1, L = tokens(i), t = first(i);
        const bool state = i > 0 || from;
        uint8_t* z = sm + b * LA_STAGE + LA_Z;
        uint8_t* out = sm + b * LA_STAGE + LA_Z;
        uint8_t* part = sm + b * LA_STAGE + LA_Y;   // SUM
        do {   // (a wait that runs out ends the walk for the whole set, below)
          if (L < LA_CH) {
            if (!(live = la_wait(&full_z[b], (i >> 1) & 1))) break;
            // rows past the document's end are another's, or none: what they hold takes no part
#pragma unroll 1
            for (int k = L * 16 + tid; k < LA_CH * 16; k += LA_SET)
              *reinterpret_cast<uint4*>(z + sw_chunk(k >> 4, k & 15, LA_CH)) = make_uint4(0u, 0u, 0u, 0u);
            fence_async_smem();
          }
          if (!(live = la_wait(&bar_qk, i & 1))) break;
          tc_fence_after();
          // Blocks of 32 columns are seen, not seen, or on the diagonal, as a warp's rows lie; 16 columns at a time, the two
          // warpgroups in turn.  P goes where the same 16 columns of QK were.  Up to 64 tokens: with what its rounding left
          // behind, in the other columns.
          const bool plain = columns && !(REV && L < LA_CH);
          auto pairs = [&](auto few) {
            constexpr bool SHORT = decltype(few)::value;
#pragma unroll 1
            for (int m = 0; m < (SHORT ? 2 : 4); ++m) {
              const int c = m * 32 + wg * 16;
              uint32_t w[8];
              float v[16];
              if (REV ? m >= quad : m <= quad) {
                tmem_ld16(tl + LT_QK + c, v);
                if (plain) {
                  const float4* near = reinterpret_cast<const float4*>(wcol + (c & 63));
                  const float2 h = m < 2 ? make_float2(1.f, 1.f) : make_float2(half, half);
#pragma unroll
                  for (int j = 0; j < 16; j += 4) {
                    const float4 n = near[j >> 2];
                    const float2 u = mul2(make_float2(v[j], v[j + 1]), mul2(make_float2(n.x, n.y), h));
                    const float2 x = mul2(make_float2(v[j + 2], v[j + 3]), mul2(make_float2(n.z, n.w), h));
                    v[j] = u.x, v[j + 1] = u.y, v[j + 2] = x.x, v[j + 3] = x.y;
                  }
                } else {
                  const int far = REV ? c - row : row - c;   // tokens between this row and the first column, or seen from it
#pragma unroll
                  for (int j = 0; j < 16; ++j) v[j] *= a.p_scale * pw[max(REV ? far + j : far - j, 0)];
                  if (REV && L < LA_CH) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                      if (c + j >= L) v[j] = 0.f;
                  }
                }
                if (m == quad) {
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    if (REV ? wg * 16 + j < lane : wg * 16 + j > lane) v[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
              } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 0u;
                if (SHORT)
#pragma unroll
                  for (int j = 0; j < 16; ++j) v[j] = 0.f;
              }
              tmem_st8(tl + LT_QK + c, w);
              if (SHORT) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  w[j] = pack_bf16(v[2 * j] - __uint_as_float(w[j] << 16), v[2 * j + 1] - __uint_as_float(w[j] & 0xffff0000u));
                tmem_st8(tl + LT_QK + LA_SHORT + c, w);
              }
            }
          };
          if (L <= LA_SHORT) pairs(std::true_type());
          else pairs(std::false_type());
          if (tid == 0 && i > 0) sent(i - 1);
          const float f = plain ? whole : back * pw[REV ? max(L - 1 - row, 0) : row + 1];
          if (state && !plain) {   // O so far is the state's: a^.. of it stays
            if (!(live = la_wait(&bar_oi[b], (i >> 1) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < 64; j += 16) {
              float v[16];
              tmem_ld16(tl + LT_O + col + j, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] *= f;
              tmem_st16(tl + LT_O + col + j, v);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          la_arrive(&bar_p);
          if (!(live = la_wait(&bar_op, i & 1) && (i >= adds || la_wait(&bar_dz[b], (i >> 1) & 1)))) break;
          tc_fence_after();
          // out by way of z, which has been read by both products (a part of a sum by y and x)
#pragma unroll 1
          for (int j = 0; j < 64; j += 32) {
            float v[32];
            if (SUM && ends && !(live = la_wait(&part_in[j >> 5][b], (i >> 1) & 1))) break;
            tmem_ld32(tl + LT_O + col + j, v);
            if (plain) {
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 u = mul2(make_float2(v[k], v[k + 1]), make_float2(f, f));
                v[k] = u.x, v[k + 1] = u.y;
              }
            }
            float4* at = reinterpret_cast<float4*>(part + la_part(row, (col + j) / 4));
            if (SUM && ends) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 n = at[k * LA_CH];
                v[4 * k] += n.x, v[4 * k + 1] += n.y, v[4 * k + 2] += n.z, v[4 * k + 3] += n.w;
              }
            }
            if (!ends) {
#pragma unroll
              for (int k = 0; k < 8; ++k) at[k * LA_CH] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(out + sw_chunk(row, (col + j) / 8 + k, LA_CH)) =
                    make_uint4(pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]),
                               pack_bf16(v[8 * k + 4], v[8 * k + 5]), pack_bf16(v[8 * k + 6], v[8 * k + 7]));
            }
          }
          tc_fence_before();
          la_arrive(&bar_o);
          fence_async_smem();
        } while (false);
        if (!(live = la_set_well<1, LA_SET>(live))) break;
        if (SUM && tid == 0) mbar_arrive(ends ? &part_empty[b] : &part_full[b]);
        if (!ends) continue;
        if (L == LA_CH) {
          if (tid == 0) {
            tma_store_3d(&a.to, out, 0, head, t);
            tma_store_3d(&a.to, out + LA_TILE / 2, 64, head, t);
            bulk_commit();
          }
        } else {   // the rows behind are another document's
#pragma unroll 1
          for (int k = tid; k < L * 16; k += LA_SET)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)(t + (k >> 4)) * a.out_token + head * D +
                                      (k & 15) * 8) = *reinterpret_cast<const uint4*>(out + sw_chunk(k >> 4, k & 15, LA_CH));
          la_set_well<1, LA_SET>(true);
        }
      }
      if (tid == 0) bulk_wait_all();
    }
  } else if (warp < 2 * LA_SET / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LA_REG_Y));
    if (OUT) make_y((tid >> 7) & 1, 2);
    else make_y(2 + ((tid >> 7) & 1), 4);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LA_REG_STATE));
    // ---- the state (held: so many times it): this thread's row y and its 64 columns z ----
    if (go_s) {
      const int me = tid - 2 * LA_SET, wg = me >> 7, quad = warp & 3, row = quad * 32 + lane, col = wg * 64;
      const uint32_t tl = tb + ((uint32_t)(quad * 32) << 16);
      uint8_t* zs = sm + LA_ZS;
      uint8_t* tile = sm + LA_STAGE;   // FP32 [128][128] for the first and the last state
      const float times = nch > 0 ? held : 1.f;   // (an empty document's passes through as it is)
      float2 S[32];
      if (from) {
        const float* src = a.init + ((int64_t)(a.init_segments ? p.segment : p.doc) * a.HV + h) * (D * D);
        if (a.init_t) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            S[j] = make_float2(times * la_load<FOLLOWS>(src + (col + 2 * j) * D + row),
                               times * la_load<FOLLOWS>(src + (col + 2 * j + 1) * D + row));
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int e = k * LA_SET + me;
            *reinterpret_cast<float4*>(tile + la_f32(e >> 5, e & 31)) = la_load<FOLLOWS>(reinterpret_cast<const float4*>(src + e * 4));
          }
          la_set_well<2, LA_SET>(true);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(tile + la_f32(row, wg * 16 + k));
            S[2 * k] = make_float2(times * v.x, times * v.y);
            S[2 * k + 1] = make_float2(times * v.z, times * v.w);
          }
          fence_async_smem();
          la_arrive(&bar_init);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = make_float2(0.f, 0.f);
      }
      auto put_state = [&] {   // as BF16
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<uint4*>(zs + sw_chunk(row, (col >> 3) + (j >> 2), D)) =
              make_uint4(pack_bf16(S[j].x, S[j].y), pack_bf16(S[j + 1].x, S[j + 1].y), pack_bf16(S[j + 2].x, S[j + 2].y),
                         pack_bf16(S[j + 3].x, S[j + 3].y));
        fence_async_smem();
        la_arrive(&bar_z);
      };
      if (OUT && nch > 0) put_state();
#pragma unroll 1
      for (int i = 0; i < adds && live; ++i) {
        if (!(live = la_wait(&bar_dz[i & 1], (i >> 1) & 1))) break;
        tc_fence_after();
        const float f = pw[tokens(i)];
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t v[16];
          tmem_ld16_async(tl + t_dz(i) + col + 2 * j, v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            S[j + k] = __ffma2_rn(make_float2(f, f), S[j + k], make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])));
        }
        tc_fence_before();
        la_arrive(&dz_read[i & 1]);
        if (OUT && i + 1 < nch) {
          if (!(live = la_wait(&bar_oi[i & 1], (i >> 1) & 1))) break;   // the state before has been used
          put_state();
        }
      }
      if (keep) {
        // by way of the other stage's y and x than the last chunk's, which have been used
        if (live && nch > 1)
          live = la_wait(&empty_y[nch & 1], ((nch - 2) >> 1) & 1) && (!OUT || la_wait(&empty_x[nch & 1], ((nch - 2) >> 1) & 1));
        const float free = columns && nch > 0 ? la_power(g, -64.f) : 1.f;
        uint8_t* way = nch > 0 && ((nch - 1) & 1) ? sm : tile;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          *reinterpret_cast<float4*>(way + la_f32(row, wg * 16 + k)) =
              make_float4(free * S[2 * k].x, free * S[2 * k].y, free * S[2 * k + 1].x, free * S[2 * k + 1].y);
        if (la_set_well<2, LA_SET>(live)) {
          float* dst = OUT ? a.last + ((int64_t)p.doc * a.HV + h) * (D * D) : a.sums + ((int64_t)p.segment * a.HV + h) * (D * D);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int e = k * LA_SET + me;
            *reinterpret_cast<float4*>(dst + e * 4) = *reinterpret_cast<const float4*>(way + la_f32(e >> 5, e & 31));
          }
        }
      }
    }
  }
  if (!live) atomicCAS(a.err, 0, ST_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == LA_MMA) tmem_dealloc(tb, 512);
  if (FOLLOWS && a.follows && blockIdx.x == gridDim.x - 1) previous_kernel_done();   // (the kernel does not end before it)
}

// Z of each segment of a document from the sums, in the walk's order; a thread takes 4 values.  Bound by the latency of its loads,
// 16 segments ahead (9 of 16 heads: 10 us alone, most of it the launch).
constexpr int LC_THREADS = 256, LC_PARTS = D * D / (4 * LC_THREADS), LC_AHEAD = 16;

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

template <bool OUT, bool REV, int TERMS, bool SUM> static cudaError_t launch_walk(const LaWalk& a, cudaStream_t s) {
  const auto kernel = la_walk_kernel<OUT, REV, TERMS, SUM>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LA_SMEM);
  if (e != cudaSuccess) return e;
  return launch_chained(kernel, dim3((unsigned)a.seg.total * a.HV), dim3(LA_THREADS), LA_SMEM, s, a);
}

cudaError_t launch_la_walk(const LaWalk& a, bool reverse, bool exact, bool sum, cudaStream_t s) {
  if (reverse) {
    if (sum) return launch_walk<true, true, 2, true>(a, s);
    return exact ? launch_walk<true, true, 3, false>(a, s) : launch_walk<true, true, 2, false>(a, s);
  }
  if (sum) return launch_walk<true, false, 2, true>(a, s);
  return exact ? launch_walk<true, false, 3, false>(a, s) : launch_walk<true, false, 2, false>(a, s);
}

cudaError_t launch_la_sums(const LaWalk& a, bool reverse, bool exact, cudaStream_t s) {
  if (reverse) return exact ? launch_walk<false, true, 3, false>(a, s) : launch_walk<false, true, 2, false>(a, s);
  return exact ? launch_walk<false, false, 3, false>(a, s) : launch_walk<false, false, 2, false>(a, s);
}

cudaError_t launch_la_carry(const LaCarry& a, cudaStream_t s) {
  return launch_chained(la_carry_kernel, dim3((unsigned)(a.seg.N * a.HV * LC_PARTS)), dim3(LC_THREADS), 0, s, a);
}

}  // namespace gdn
