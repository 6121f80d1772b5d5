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

constexpr int QK_THREADS = 128;
constexpr int QK_WARPS = QK_THREADS / 32;
constexpr int QK_MAXD = 512;        // any layout
constexpr int QK_FAST_MAXD = 256;   // rows of pieces of 8 values
constexpr int QK_STEPS = 16;
constexpr int QK_CTAS = 64;         // CTAs per SM of a grid that walks its work, at most

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
  // the work (divide_work): CTAs 0 .. ctas_q-1 take q, the others k; a unit is `run` heads of as many
  // neighbouring tokens as a warp has rows
  int run, splits[2], units[2], ctas_q;
};

// f / 2 pi, the turns per position, as a fraction of 2^64 (modulo whole turns): f's 53-bit mantissa times
// 2^66 / 2 pi, shifted by its exponent, in integers, since FP64 arithmetic is slow here and a single token's call waits for it
__device__ __forceinline__ uint64_t turn_step(double f) {
  constexpr uint64_t PER_TURN = 0xA2F9836E4E441529ull;   // floor(2^66 / 2 pi)
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)(bits >> 52) & 0x7ff;
  if (e == 0) return 0;   // zero, or less than 2^-1022
  const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  const uint64_t hi = __umul64hi(m, PER_TURN), lo = m * PER_TURN;
  const int down = 1077 - e;   // f = m 2^(e - 1075), and the product counts 2^-66 turns: down to 2^-64
  const uint64_t t = down >= 128 ? 0 : down >= 64 ? hi >> (down - 64)
                     : down > 0 ? (hi << (64 - down)) | (lo >> down) : down > -64 ? lo << -down : 0;
  return bits >> 63 ? 0 - t : t;
}
// m cos and m sin at position pos. FAST: within 2^-20, by the hardware's functions, for 16-bit rows, whose values are then
// rounded to 8 or 11 bits. The FP32 sums dwq and dwk of such rows are not, but their terms' errors are of either sign and add
// up like the sum's own roundings: 32,768 tokens of 16 + 16 heads of 128, BF16, 2.1e-7 of the norm from FP64 (FP32 rows,
// by sincospif, 1.9e-7; elementary FP32 operations 4.6e-7), 300 tokens of 8 + 2 heads 1.8e-7 (operations 1.5e-7).
template <bool FAST>
__device__ __forceinline__ void angle_cos_sin(uint64_t step, int pos, float m, float* c, float* s) {
  const uint64_t turn = step * (uint64_t)(int64_t)pos;
  const float part = (float)(int)(uint32_t)(turn >> 32);   // of 2^32 a turn: within half a turn
  if (FAST) {
    const float angle = part * (3.14159265358979f / 2147483648.f);
    *c = __cosf(angle);
    *s = __sinf(angle);
  } else {
    sincospif(part * (1.f / 2147483648.f), s, c);
  }
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

// ---- rows of the fast kernels ----
// A row lies in pieces of 8 values, two blocks of 4: L lanes have M pieces each, the pieces l, l + L, .. of lane l.  In the
// half layout a piece's blocks are partners, 4 values of the first rotated half and the 4 they are turned with, so that
// no value crosses lanes; pieces past the rotated part, and all of the pairs layout, have 8 neighbouring values.  Where the
// rotated part is 4 and a multiple of 8, that goes for each half of a piece by itself (HALF_BY_4: 100,000 tokens of 16 + 4
// heads of 80, 20 rotated, forward 186 us and backward 283; the kernel for any rows 346 and 588).  Either way pairs 4i .. 4i+3
// are piece i's.
// Values are held as 4 float2: v[j] has the partner v[j ^ 2] (half), or its own other value (pairs).
enum { PAIRS = 0, HALF = 1, HALF_BY_4 = 2 };
template <int L, int M, int LAYOUT> struct Pieces {
  static constexpr int B = LAYOUT == HALF_BY_4 ? 2 : 1;   // parts of a piece
  int off[M][B], away[M][B];   // of a part's first block, and from there to the second
  int rotated[M];              // how many of the piece's values are
  bool has[M];                 // the row is so long
  __device__ __forceinline__ void setup(const QkArgs& a, int l) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int i = l + m * L;
      rotated[m] = LAYOUT == PAIRS ? a.rot - 8 * i : 0;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int e = B * i + b;
        const bool apart = LAYOUT != PAIRS && e < a.rot * B / 8;   // (whole parts: those before hold rot values)
        off[m][b] = (apart ? 4 : 8) / B * e;
        away[m][b] = apart ? a.rot / 2 : 4 / B;
        if (apart) rotated[m] += 8 / B;
      }
      has[m] = i < a.D / 8;
    }
  }
  // of v[j]
  __device__ __forceinline__ int place(int m, int j) const {
    return B == 2 ? off[m][j & (B - 1)] + (j < 2 ? 0 : away[m][j & (B - 1)]) : off[m][0] + (j < 2 ? 0 : away[m][0]) + (j & 1) * 2;
  }
  // v with zeros where nothing is rotated: an infinite value's neighbour must not take part, not even times a zero sine
  __device__ __forceinline__ void only_rotated(int m, float2 (&v)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((LAYOUT == HALF_BY_4 ? 4 * (j & 1) : 2 * j) >= rotated[m]) v[j] = make_float2(0.f, 0.f);
  }
};

template <typename E> __device__ __forceinline__ float2 pair_at(const uint32_t* u, int j) {
  if constexpr (sizeof(E) == 4) return make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
  else return pair_f32(u[j], (const E*)nullptr);
}

// piece m of the row at `row` + PAST bytes in shared memory
template <typename E, int PAST, int L, int M, int LAYOUT>
__device__ __forceinline__ void read_piece(uint32_t row, const Pieces<L, M, LAYOUT>& p, int m, float2 (&v)[4]) {
  if constexpr (LAYOUT == HALF_BY_4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      RawV<E, 2> r;
      r.load_shared(row + p.place(m, j) * (int)sizeof(E) + PAST);
      v[j] = pair_at<E>(r.u, 0);
    }
    return;
  }
  const uint32_t at = row + p.off[m][0] * (int)sizeof(E) + PAST;   // (PAST here: the backward 946 us, at the loads 954)
  RawV<E, 4> b[2];
  if constexpr (LAYOUT == PAIRS && sizeof(E) == 2) {
    RawV<E, 8> r;
    r.load_shared(at);
    b[0].u[0] = r.u[0];
    b[0].u[1] = r.u[1];
    b[1].u[0] = r.u[2];
    b[1].u[1] = r.u[3];
  } else {
    b[0].load_shared(at);
    b[1].load_shared(at + p.away[m][0] * (int)sizeof(E));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pair_at<E>(b[j >> 1].u, j & 1);
}
template <typename E, int L, int M, int LAYOUT>
__device__ __forceinline__ void write_piece(E* row, const Pieces<L, M, LAYOUT>& p, int m, const float2 (&v)[4]) {
  if constexpr (LAYOUT == HALF_BY_4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      RawV<E, 2> r;
      const float f[2] = {v[j].x, v[j].y};
      r.put(f);
      r.store(row + p.place(m, j));
    }
    return;
  }
  E* at = row + p.off[m][0];
  RawV<E, 4> b[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float f[4] = {v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y};
    b[j].put(f);
  }
  if constexpr (LAYOUT == PAIRS && sizeof(E) == 2) {
    RawV<E, 8> r;
    r.u[0] = b[0].u[0];
    r.u[1] = b[0].u[1];
    r.u[2] = b[1].u[0];
    r.u[3] = b[1].u[1];
    r.store(at);
  } else {
    b[0].store(at);
    b[1].store(at + p.away[m][0]);
  }
}

// Rows on their way to a warp: a ring of STAGES slots of its own shared memory, each the 32 / L rows of one step of
// the warp (of N tensors). The warp's lanes copy 16 bytes at a time, so that the bytes in flight cost no registers.
template <typename E, int L, int N, int M> struct Ring {
  static constexpr int CHUNKS = M * (int)sizeof(E) / 2;          // 16-byte chunks a lane copies of a row
  static constexpr int ROW = 8 * L * M;                              // values a row has room for
  static constexpr int ROWS = 32 / L;
  static constexpr int SLOT = N * ROWS * ROW;                    // values
  static constexpr int BYTES = SLOT * (int)sizeof(E);
  static __device__ __forceinline__ int next(int at) { return at + BYTES == STAGES * BYTES ? 0 : at + BYTES; }
  static constexpr int STAGES = N * CHUNKS == 1 ? 8 : N * CHUNKS == 2 ? 6 : N * CHUNKS < 6 ? 4 : 3;
};
// Values of a row past D are never copied, and are zero from the start.
template <typename E, int L, int N, int M> __device__ __forceinline__ void clear_ring(E* slots, int D) {
  using R = Ring<E, L, N, M>;
  if (D == R::ROW) return;
  for (int i = threadIdx.x & 31; i < R::STAGES * R::SLOT / R::ROW * (R::ROW - D); i += 32) {
    const int row = i / (R::ROW - D);
    slots[row * R::ROW + D + i - row * (R::ROW - D)] = from_f32<E>(0.f);
  }
  __syncwarp();
}
__device__ __forceinline__ void copy16(uint32_t smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(global) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

template <int LAYOUT> __device__ __forceinline__ float2 partner_of(const float2 (&v)[4], int j) {
  return LAYOUT != PAIRS ? v[j ^ 2] : make_float2(v[j].y, v[j].x);
}

// A lane's pairs, four a piece: their turn steps, and cos and sin at a token laid out like the lane's values,
// y[j] = v[j] co[j] + partner[j] si[j].  Pairs past the rotated part get the identity.
template <int L, int M, int LAYOUT, bool FAST> struct Angles {
  uint64_t step[M][4];
  double f[M][4];
  // the frequencies are requested first, and converted when the rows' copies are on their way
  __device__ __forceinline__ void request(const QkArgs& a, int l) {
#pragma unroll
    for (int i = 0; i < 4 * M; ++i) {
      const int p = 4 * (l + i / 4 * L) + i % 4;
      f[i / 4][i % 4] = p < a.rot / 2 ? a.freq[p] : 0.0;
    }
  }
  __device__ __forceinline__ void setup() {
#pragma unroll
    for (int i = 0; i < 4 * M; ++i) step[i / 4][i % 4] = turn_step(f[i / 4][i % 4]);
  }
  // of piece m
  __device__ __forceinline__ void at(const QkArgs& a, int pos, int l, int m, float2 (&co)[4], float2 (&si)[4]) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      angle_cos_sin<FAST>(step[m][i], pos, a.mscale, &c[i], &s[i]);
      if (4 * (l + m * L) + i >= a.rot / 2) {
        c[i] = 1.f;
        s[i] = 0.f;
      }
    }
    if (LAYOUT != PAIRS) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        co[j] = co[j + 2] = make_float2(c[2 * j], c[2 * j + 1]);
        si[j] = make_float2(-s[2 * j], -s[2 * j + 1]);
        si[j + 2] = make_float2(s[2 * j], s[2 * j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        co[j] = make_float2(c[j], c[j]);
        si[j] = make_float2(-s[j], s[j]);
      }
    }
  }
};

// A warp's place in its work on one kind of heads: one token for each group of L lanes, `run` heads of them. A group past
// the last token works on the last one, and keeps nothing.
template <int L> struct Place {
  int unit, h, left;   // left: heads of the run from h on
  int64_t t;
  bool live;
  __device__ __forceinline__ void enter(const QkArgs& a, int splits, int heads) {
    int tokens = unit, part = 0;
    if (splits > 1) {
      tokens = unit / splits;
      part = unit - tokens * splits;
    }
    t = (int64_t)tokens * (32 / L) + (threadIdx.x & 31) / L;
    live = t < a.T;
    t = live ? t : a.T - 1;
    h = part * a.run;
    left = min(a.run, heads - h);
  }
};

// The weights of piece m (zeros where there is none)
template <int L, int M, int LAYOUT>
__device__ __forceinline__ void piece_weights(const float* w, const Pieces<L, M, LAYOUT>& p, int m, float2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = p.place(m, j);
    v[j] = !p.has[m] ? make_float2(0.f, 0.f) : w ? make_float2(w[d], w[d + 1]) : make_float2(1.f, 1.f);
  }
}

template <int L> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int x = L / 2; x >= 1; x >>= 1) v += __shfl_xor_sync(~0u, v, x);
  return v;
}

// ---- rows of any kind, value by value: lane i has the values i, i + 32, ... ----
template <int PER> struct RowAngles {
  float c[PER], s[PER];   // value = value c + partner s
  int partner[PER];
  int doc = 0;
  uint64_t step[PER];
  __device__ __forceinline__ void setup(const QkArgs& a) {
    const int half = a.rot / 2;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int d = (threadIdx.x & 31) + 32 * i;
      partner[i] = a.half_layout ? (d < half ? d + half : d - half) : d ^ 1;
      step[i] = d < a.rot ? turn_step(a.freq[a.half_layout ? (d < half ? d : d - half) : d >> 1]) : 0;
    }
  }
  __device__ __forceinline__ void at(const QkArgs& a, int64_t t) {
    const int pos = position_of(a, t, &doc);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int d = (threadIdx.x & 31) + 32 * i;
      if (d >= a.rot) break;
      angle_cos_sin<false>(step[i], pos, a.mscale, &c[i], &s[i]);
      if (d < partner[i]) s[i] = -s[i];
    }
  }
};
template <int PER> __device__ __forceinline__ void row_weights(const float* w, int D, float (&v)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int d = (threadIdx.x & 31) + 32 * i;
    v[i] = d >= D ? 0.f : w ? w[d] : 1.f;
  }
}

// rows without masks: normed and rotated whole
inline bool plain_rows(const QkArgs& a) { return a.normed && a.rot == a.D; }

// 16-bit rows of 9 .. 12 and of 17 .. 24 pieces, which would leave up to half of 16 or 32 lanes without any, lie in 4 and 8 lanes
// of three: their kernels would be bound by instructions (100,000 tokens of 16 + 4 heads of 96: forward 120 us, with one
// piece a lane 149, backward 191 and 230; FP32 rows reach the copy rate as they are).  Not so a few rows, for which a
// lane's own work is all (one token 3.05 and 2.64 us; 64: 3.17 and 3.16; 300: 3.79 and 4.90).
inline bool three_pieces(const QkArgs& a) { return a.T * (a.heads[0] + a.heads[1]) >= 8 * sm_count(); }

// Divides the work: runs of heads as long as the warps that the GPU holds at once (`resident` CTAs an SM) get `least`
// units each; then a whole number of such rounds of CTAs, so that SMs that are ahead take more of them (262,144
// tokens of 16 + 16 heads, forward: one round 741 us, three 662, ten 633), as long as a warp has least * QK_STEPS rows a
// group for its start (74,155 tokens of 1 + 1 heads of 64, forward: 14 us against 25); and q's and k's shares by their heads. least
// is 1 for the forward and, since every CTA leaves partial sums to add, 2 for the backward (32,768 tokens, forward: 82 us
// with 1, 97 with 4; backward 139 with 1, 130 with 2, 133 with 4).  Returns the CTAs.
inline int divide_work(QkArgs& a, int L, int resident, int least) {
  const int total = a.heads[0] + a.heads[1], rows = 32 / L;
  const int64_t round = (int64_t)sm_count() * (resident < 1 ? 1 : resident);
  const int64_t groups = (a.T + rows - 1) / rows, most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
  int64_t run = groups * total / (round * QK_WARPS * least);
  run = run < 1 ? 1 : run > most ? most : run;
  a.run = (int)run;
  int64_t ctas = 0;
  for (int i = 0; i < 2; ++i) {
    a.splits[i] = (a.heads[i] + a.run - 1) / a.run;
    a.units[i] = (int)(groups * a.splits[i]);   // (below 2^31: splits are 1 unless tokens are few)
    ctas += (a.units[i] + QK_WARPS - 1) / QK_WARPS;
  }
  int64_t rounds = groups * total / (round * QK_WARPS * QK_STEPS * least);
  rounds = rounds < 1 ? 1 : rounds > 10 ? 10 : rounds;
  const int64_t limit = round * rounds < (int64_t)sm_count() * QK_CTAS ? round * rounds : (int64_t)sm_count() * QK_CTAS;
  if (ctas > limit) ctas = limit;
  a.ctas_q = (int)((ctas * a.heads[0] + total / 2) / total);
  if (a.heads[0] > 0 && a.heads[1] > 0) {
    if (ctas < 2) ctas = 2;
    a.ctas_q = a.ctas_q < 1 ? 1 : a.ctas_q > ctas - 1 ? (int)ctas - 1 : a.ctas_q;
  }
  return (int)ctas;
}
// CTAs an SM holds of a kernel, asked once
template <typename K> inline int resident_ctas(K kernel) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, QK_THREADS, 0) != cudaSuccess) n = 1;
  return n;
}

// --- gdn_qk_bwd.cu ---
void launch_qk_bwd(QkArgs& a, int dtype, bool fast, float* dwq, float* dwk, cudaStream_t s);

}  // namespace gdn
