// gdn_step_tables.cu -- the tables of a generation step from the requests' lengths, on the GPU.
//
// The states of a request lie in blocks of B tokens: block j's slot holds the state after the last of the tokens
// jB .. (j+1)B - 1 that has been taken.  All of it is sums over the requests in their order (tokens taken, blocks needed,
// blocks given back) and then one write a token, so it is one kernel of one cluster: every CTA works the sums out
// for itself in shared memory, and they share the writes.  Bound by the latency of its few dependent steps (64 requests of a
// token each: 5.4 us).  Where tokens are many, a second kernel writes theirs from the first one's tables (2,000 requests, 60,000
// tokens; by the one cluster 21 us).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_prof.h"

namespace gdn {

constexpr int TB_THREADS = 1024, TB_MOST = 16384;   // threads of a CTA; requests
constexpr int TB_SMALL = 256;      // threads where requests and tokens are no more than that (64 of a token: 4.1 us, by 1,024 5.2)
constexpr int TB_KEPT = 8192;      // so many requests' lengths and contexts are kept in shared memory, too
constexpr int TB_CLUSTER = 8;      // CTAs where there is more to write than
// So many tokens or requests; beyond it the tokens are a second kernel's (1,000 requests of a token: 7.6 us, by two kernels 9.5;
// 64 of 32 7.6 and 8.3, of 60 9.3 and 8.4; 4,000 of one 20 and 16)
constexpr int TB_ALONE = 2048;

struct StepTableArgs {
  const int* lengths;
  const int* context;
  int* context_out;
  int* blocks;
  int* free_list;
  const int* free_count;
  int* free_count_out;
  int* cu;
  int* positions;
  int* slot_in;
  int* slot_out;
  int* err;
  int N, T, block, row, slots;
  int apart;   // the tokens' tables are the second kernel's
};

struct Request {
  int take, held, need, back;   // tokens; blocks held, needed, given back
};

__device__ __forceinline__ Request request_of(const StepTableArgs& a, int len, int ctx, bool* bad) {
  Request r = {0, 0, 0, 0};
  const int64_t after = (int64_t)ctx + max(len, 0);
  if (len < -1 || ctx < 0 || after > (int64_t)a.row * a.block) {
    *bad = true;
    return r;
  }
  r.held = (int)(((int64_t)ctx + a.block - 1) / a.block);
  if (len < 0) {
    r.back = r.held;
  } else {
    r.take = len;
    r.need = (int)((after + a.block - 1) / a.block) - r.held;
  }
  return r;
}

// the request whose part of a running sum (sum[n] <= e < sum[n + 1]) the element e is
__device__ __forceinline__ int owner_of(const int* sum, int N, int e) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

// position and slot of token t of request n, whose tokens end before `end`; first: its position is t more than that
__device__ __forceinline__ void write_token(const StepTableArgs& a, int t, int tokens, int n, int first, int end) {
  int pos = 0, slot = -1;
  if (t < tokens) {
    pos = first + t;
    if (t == end - 1 || pos % a.block == a.block - 1) slot = __ldcg(a.blocks + (int64_t)n * a.row + pos / a.block);
  }
  if (a.positions) a.positions[t] = pos;
  a.slot_out[t] = slot;
}

// the tokens' tables from the requests': a request that has taken tokens had so many fewer before
__global__ void __launch_bounds__(TB_THREADS) step_tokens_kernel(const StepTableArgs a) {
  chain_kernel();
  extern __shared__ int tb_smem[];
  const int* cu = a.cu;
  if (a.N <= TB_KEPT) {
    for (int n = threadIdx.x; n <= a.N; n += blockDim.x) tb_smem[n] = __ldcg(a.cu + n);
    __syncthreads();
    cu = tb_smem;
  }
  const int tokens = cu[a.N];
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < a.T; t += gridDim.x * blockDim.x) {
    const int n = t < tokens ? owner_of(cu, a.N, t) : 0;
    const int end = t < tokens ? cu[n + 1] : 0;
    write_token(a, t, tokens, n, t < tokens ? __ldcg(a.context_out + n) - end : 0, end);
  }
}

__global__ void __launch_bounds__(TB_THREADS) step_tables_kernel(const StepTableArgs a) {
  chain_kernel();
  namespace cg = cooperative_groups;
  extern __shared__ int tb_smem[];
  int *start = tb_smem, *fresh = start + a.N + 1, *given = fresh + a.N + 1;   // tokens, new blocks, returned blocks before
  __shared__ int64_t words[3][32];
  __shared__ int first_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int me = rank * blockDim.x + threadIdx.x, all = ctas * blockDim.x;
  const int *lengths = a.lengths, *context = a.context;
  if (a.N <= TB_KEPT) {
    int *l = given + a.N + 1, *c = l + a.N;
    for (int n = threadIdx.x; n < a.N; n += blockDim.x) l[n] = a.lengths[n], c[n] = a.context[n];   // (read again by the same thread first)
    lengths = l;
    context = c;
  }
  bool bad = false;
  int64_t held = *a.free_count;
  if (held < 0 || held > a.slots) {
    bad = true;
    held = 0;
  }
  if (threadIdx.x == 0) start[0] = fresh[0] = given[0] = 0, first_s = a.N;
  // running sums of the tokens, the blocks needed and the blocks that come back (past 2^31, as much: it fits nowhere)
  int64_t before[3] = {0, 0, 0};
  for (int n0 = 0; n0 < a.N; n0 += blockDim.x) {
    const int n = n0 + threadIdx.x;
    const Request r = n < a.N ? request_of(a, lengths[n], context[n], &bad) : Request{0, 0, 0, 0};
    int64_t v[3] = {r.take, r.need, r.back};
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, v[i], d);
        if (lane >= d) v[i] += x;
      }
    __syncthreads();
    if (lane == 31)
      for (int i = 0; i < 3; ++i) words[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      int64_t w = lane < warps ? words[i][lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, w, d);
        if (lane >= d) w += x;
      }
      const int64_t up = __shfl_sync(~0u, w, (warp + 31) & 31), total = __shfl_sync(~0u, w, 31);
      v[i] += before[i] + (warp ? up : 0);
      before[i] += total;
    }
    if (n < a.N) {
      start[n + 1] = (int)min(v[0], (int64_t)INT32_MAX);
      fresh[n + 1] = (int)min(v[1], (int64_t)INT32_MAX);
      given[n + 1] = (int)min(v[2], (int64_t)INT32_MAX);
    }
  }
  int64_t back = before[2];
  if (held + back > a.slots) {   // (more than there are: some were not this pool's)
    bad = true;
    back = a.slots - held;
  }
  const int64_t top = held + back;
  if (bad && rank == 0) *a.err = ST_DEVICE;
  __syncthreads();
  // The first request that does not fit, and all after it, wait.
  if (before[0] > a.T || before[1] > top) {
    for (int n = threadIdx.x; n < a.N; n += blockDim.x)
      if (start[n + 1] > a.T || fresh[n + 1] > top) atomicMin(&first_s, n);
    __syncthreads();
    const int fit = first_s, t = start[fit], f = fresh[fit];
    __syncthreads();
    for (int n = fit + threadIdx.x; n < a.N; n += blockDim.x) start[n + 1] = t, fresh[n + 1] = f;
    __syncthreads();
  }
  const int tokens = start[a.N], taken = fresh[a.N];
  // returned blocks on top of the free ones
  if (back > 0) {
    for (int e = me; e < back; e += all) {
      const int n = owner_of(given, a.N, e);
      a.free_list[held + e] = a.blocks[(int64_t)n * a.row + (e - given[n])];
    }
    cluster.sync();
  }
  // new ones from there
  if (taken > 0) {
    for (int e = me; e < taken; e += all) {
      const int n = owner_of(fresh, a.N, e);
      const int held_n = (int)(((int64_t)context[n] + a.block - 1) / a.block);
      a.blocks[(int64_t)n * a.row + held_n + (e - fresh[n])] = __ldcg(a.free_list + (top - 1 - e));
    }
    cluster.sync();
  }
  for (int n = me; n < a.N; n += all) {
    bool b = false;
    const int ctx = context[n];
    const Request r = request_of(a, lengths[n], ctx, &b);
    a.slot_in[n] = r.held > 0 && r.back == 0 ? __ldcg(a.blocks + (int64_t)n * a.row + (ctx - 1) / a.block) : -1;
    a.cu[n + 1] = start[n + 1];
  }
  if (me == 0) a.cu[0] = 0;
  if (!a.apart) {
    for (int t = me; t < a.T; t += all) {
      const int n = t < tokens ? owner_of(start, a.N, t) : 0;
      write_token(a, t, tokens, n, t < tokens ? context[n] - start[n] : 0, t < tokens ? start[n + 1] : 0);
    }
  }
  cluster.sync();   // all has been read: the books may be the ones that go on
  for (int n = me; n < a.N; n += all) {
    bool b = false;
    const int len = lengths[n], ctx = context[n];
    request_of(a, len, ctx, &b);
    a.context_out[n] = len == -1 && !b ? 0 : ctx + start[n + 1] - start[n];
  }
  if (me == 0) *a.free_count_out = (int)top - taken;
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_step_tables(const gdn_tables_problem* p, const int32_t* lengths, const int32_t* context,
                                      int32_t* context_out, int32_t* blocks, int32_t* free_list, const int32_t* free_count,
                                      int32_t* free_count_out, int32_t* cu, int32_t* positions, int32_t* slot_in,
                                      int32_t* slot_out, int32_t* err, struct CUstream_st* stream) {
  if (!p || p->N < 0 || p->T < 0 || p->block < 1 || p->max_blocks < 0 || p->slots < 0) return GDN_ERR_INVALID_ARG;
  if (p->N > TB_MOST || p->T > INT32_MAX / 2 || (int64_t)p->max_blocks * p->block > INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !cu || !err || !on_words(free_count, free_count_out, cu, err)) return GDN_ERR_INVALID_ARG;
  if (p->N > 0 && (!lengths || !context || !context_out || !slot_in)) return GDN_ERR_INVALID_ARG;
  if ((p->N > 0 && p->max_blocks > 0 && !blocks) || (p->slots > 0 && !free_list) || (p->T > 0 && !slot_out)) return GDN_ERR_INVALID_ARG;
  if (!on_words(lengths, context, context_out, blocks, free_list, positions, slot_in, slot_out)) return GDN_ERR_INVALID_ARG;
  const StepTableArgs a = {lengths, context, context_out, blocks, free_list, free_count, free_count_out, cu, positions, slot_in,
                           slot_out, err, p->N, p->T, p->block, p->max_blocks, p->slots, p->T > TB_ALONE};
  const int bytes = ((p->N <= TB_KEPT ? 5 : 3) * p->N + 3) * (int)sizeof(int);
  static_assert(3 * TB_MOST >= 5 * TB_KEPT, "the larger need is what is asked for");
  if (cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (3 * TB_MOST + 3) * (int)sizeof(int)) !=
      cudaSuccess)
    return GDN_ERR_CUDA;
  const int ctas = p->T > TB_ALONE || p->N > TB_ALONE ? TB_CLUSTER : 1;
  const int threads = p->T <= TB_SMALL && p->N <= TB_SMALL ? TB_SMALL : TB_THREADS;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  prof_begin(K_STEP_TABLES, stream);
  cudaError_t e = cudaLaunchKernelEx(&cfg, step_tables_kernel, a);
  if (e == cudaSuccess && a.apart) {
    const int need = (p->T + TB_THREADS - 1) / TB_THREADS, most = 2 * sm_count();
    e = launch_chained(step_tokens_kernel, dim3(need < most ? need : most), dim3(TB_THREADS),
                       p->N <= TB_KEPT ? (p->N + 1) * sizeof(int) : 0, stream, a);
  }
  prof_end(K_STEP_TABLES, stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
