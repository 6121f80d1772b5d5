// gdn_step_tables.cu -- the tables of a generation step from the requests' lengths, on the GPU.
//
// The states of a request lie in blocks of B tokens: block j's slot holds the state after the last of the tokens
// jB .. (j+1)B - 1 that has been taken.  All of it is sums over the requests in their order (tokens taken, blocks needed,
// blocks given back) and then one write a token, so it is one kernel of one cluster: every CTA works the sums out
// for itself in shared memory, and they share the writes.  Bound by the latency of its few dependent steps.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_prof.h"

namespace gdn {

constexpr int TB_THREADS = 1024, TB_MOST = 16384;   // requests
constexpr int TB_CLUSTER = 8;      // CTAs where there is more to write than
constexpr int TB_ALONE = 4096;     // so many tokens and blocks

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
};

struct Request {
  int take, held, need, back;   // tokens; blocks held, needed, given back
};

__device__ __forceinline__ Request request_of(const StepTableArgs& a, int n, bool* bad) {
  Request r = {0, 0, 0, 0};
  const int len = a.lengths[n], ctx = a.context[n];
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

// inclusive sums over the CTA's threads; `total` of all of them
__device__ __forceinline__ int64_t over_cta(int64_t v, int64_t* words, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, v, d);
    if (lane >= d) v += x;
  }
  __syncthreads();
  if (lane == 31) words[warp] = v;
  __syncthreads();
  int64_t w = words[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, w, d);
    if (lane >= d) w += x;
  }
  *total = __shfl_sync(~0u, w, 31);
  const int64_t before = __shfl_sync(~0u, w, (warp + 31) & 31);
  return v + (warp ? before : 0);
}

__global__ void __launch_bounds__(TB_THREADS) step_tables_kernel(const StepTableArgs a) {
  chain_kernel();
  namespace cg = cooperative_groups;
  extern __shared__ int tb_smem[];
  int *start = tb_smem, *fresh = start + a.N + 1, *given = fresh + a.N + 1;   // tokens, new blocks, returned blocks before
  __shared__ int64_t words[3][32];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int lane = threadIdx.x & 31, warp = rank * (TB_THREADS / 32) + (threadIdx.x >> 5), warps = ctas * (TB_THREADS / 32);
  bool bad = false;
  int64_t held = *a.free_count;
  if (held < 0 || held > a.slots) {
    bad = true;
    held = 0;
  }
  // blocks that come back
  int64_t back = 0, take = 0, need = 0, all;
  for (int n0 = 0; n0 < a.N; n0 += TB_THREADS) {
    const int n = n0 + threadIdx.x;
    const Request r = n < a.N ? request_of(a, n, &bad) : Request{0, 0, 0, 0};
    const int64_t sum = over_cta(r.back, words[0], &all);
    if (n < a.N) given[n] = (int)min(back + sum - r.back, (int64_t)INT32_MAX);
    back += all;
  }
  if (held + back > a.slots) {   // (more than there are: some were not this pool's)
    bad = true;
    back = a.slots - held;
  }
  const int64_t top = held + back;
  // Those that fit take their tokens and blocks: the first that does not, and all after it, wait.  The sums only
  // grow, so each request sees for itself.
  for (int n0 = 0; n0 < a.N; n0 += TB_THREADS) {
    const int n = n0 + threadIdx.x;
    const Request r = n < a.N ? request_of(a, n, &bad) : Request{0, 0, 0, 0};
    const int64_t st = over_cta(r.take, words[1], &all) + take;
    take += all;
    const int64_t sn = over_cta(r.need, words[2], &all) + need;
    need += all;
    const bool fits = st <= a.T && sn <= top;
    // (of those that wait, the sums before them, which no later one passes: what the last that fits leaves)
    if (n < a.N) {
      start[n + 1] = fits ? (int)st : -1;
      fresh[n + 1] = fits ? (int)sn : -1;
    }
  }
  if (threadIdx.x == 0) start[0] = fresh[0] = 0;
  __syncthreads();
  // the first that waits, by the sums that were not kept
  __shared__ int first_s;
  if (threadIdx.x == 0) first_s = a.N;
  __syncthreads();
  for (int n = threadIdx.x; n < a.N; n += TB_THREADS)
    if (start[n + 1] < 0) atomicMin(&first_s, n);
  __syncthreads();
  const int fit = first_s;
  const int tokens = start[fit], taken = fresh[fit];
  __syncthreads();
  for (int n = fit + threadIdx.x; n < a.N; n += TB_THREADS) {
    start[n + 1] = tokens;
    fresh[n + 1] = taken;
  }
  __syncthreads();
  if (bad && rank == 0) *a.err = ST_DEVICE;
  // returned blocks on top of the free ones
  for (int n = warp; n < a.N; n += warps) {
    bool b = false;
    const Request r = request_of(a, n, &b);
    const int64_t at = held + given[n];
    for (int j = lane; j < r.back; j += 32)
      if (at + j < a.slots) a.free_list[at + j] = a.blocks[(int64_t)n * a.row + j];
  }
  cluster.sync();
  // new ones from there
  for (int n = warp; n < a.N; n += warps) {
    const int count = fresh[n + 1] - fresh[n];
    if (count <= 0) continue;
    bool b = false;
    const Request r = request_of(a, n, &b);
    for (int j = lane; j < count; j += 32)
      a.blocks[(int64_t)n * a.row + r.held + j] = __ldcg(a.free_list + (top - 1 - fresh[n] - j));
  }
  cluster.sync();
  for (int n = rank * TB_THREADS + threadIdx.x; n < a.N; n += ctas * TB_THREADS) {
    const int ctx = a.context[n];
    bool b = false;
    const Request r = request_of(a, n, &b);
    a.slot_in[n] = r.held > 0 && r.back == 0 ? __ldcg(a.blocks + (int64_t)n * a.row + (ctx - 1) / a.block) : -1;
    a.cu[n + 1] = start[n + 1];
  }
  if (rank == 0 && threadIdx.x == 0) a.cu[0] = 0;
  for (int t = rank * TB_THREADS + threadIdx.x; t < a.T; t += ctas * TB_THREADS) {
    int pos = 0, slot = -1;
    if (t < tokens) {
      int lo = 0, hi = a.N;   // start[lo] <= t < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid;
      }
      pos = a.context[lo] + t - start[lo];
      if (t == start[lo + 1] - 1 || pos % a.block == a.block - 1) slot = __ldcg(a.blocks + (int64_t)lo * a.row + pos / a.block);
    }
    if (a.positions) a.positions[t] = pos;
    a.slot_out[t] = slot;
  }
  cluster.sync();   // all has been read: the books may be the ones that go on
  for (int n = rank * TB_THREADS + threadIdx.x; n < a.N; n += ctas * TB_THREADS) {
    bool b = false;
    request_of(a, n, &b);
    a.context_out[n] = a.lengths[n] == -1 && !b ? 0 : a.context[n] + start[n + 1] - start[n];
  }
  if (rank == 0 && threadIdx.x == 0) *a.free_count_out = (int)top - taken;
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
                           slot_out, err, p->N, p->T, p->block, p->max_blocks, p->slots};
  const int bytes = (3 * p->N + 3) * (int)sizeof(int);
  if (cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (3 * TB_MOST + 3) * (int)sizeof(int)) !=
      cudaSuccess)
    return GDN_ERR_CUDA;
  const int ctas = p->T > TB_ALONE || p->N > TB_ALONE ? TB_CLUSTER : 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(TB_THREADS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  prof_begin(K_STEP_TABLES, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, step_tables_kernel, a);
  prof_end(K_STEP_TABLES, stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
