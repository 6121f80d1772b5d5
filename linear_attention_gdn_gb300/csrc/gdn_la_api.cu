// gdn_la_api.cu -- host layer of the linear attention: checks, the cut into segments, and the walks of each entry point.
#include <algorithm>
#include <cstring>

#include "gdn.h"
#include "gdn_elem.cuh"
#include "gdn_internal.h"
#include "gdn_la.cuh"
#include "gdn_prof.h"

namespace gdn {

bool make_tmap_strided(CUtensorMap* m, const void* base, int64_t T, int heads, int64_t token, int rows);

constexpr double LA_BEGIN = 2.2;   // of a walk, in chunks

struct LaPlan {
  int len, total;   // chunks of a segment, segments
  bool split;       // some document has more than one
  uint64_t bounds;  // of the table, as the kernels compare it
};

static int chunks_of(const int32_t* cu, int d) { return (int)(((int64_t)cu[d + 1] - cu[d] + LA_CH - 1) / LA_CH); }

static int64_t segments_of(const gdn_la_problem* p, const int32_t* cu, int len) {
  int64_t n = 0;
  for (int d = 0; d < p->N; ++d) n += std::max(1, (chunks_of(cu, d) + len - 1) / len);
  return n;
}

// The cut into segments.  A walk of one segment and head is a CTA, one to an SM; its time is its chunks (2.5 us each) and what
// begins and ends it (5.4 us).  Cutting costs a second pass over two of the four tensors, about 0.8 of the walk, and the carry
// between.  So documents stay whole unless the longest is the better part of the time, and then the number of pieces is
// taken for which the rounds of CTAs are estimated to end first (one document of 32,768 tokens and 16 heads: whole 668 us, in 19
// pieces, two rounds of CTAs, 179, in 9, one round, 157; of 8,192 and 48 heads: whole 178, in 3 pieces 124, in 8 161; of 2,048:
// whole 53, in 2 pieces 63).
static gdn_status la_plan(const gdn_la_problem* p, const int32_t* cu, LaPlan* plan) {
  if (!p || !cu) return GDN_ERR_INVALID_ARG;
  if (p->N < 1 || p->T < 0 || p->H < 1 || p->HV < 1 || p->segment < 0) return GDN_ERR_INVALID_ARG;
  if (p->dk != 128 || p->dv != 128 || p->HV % p->H != 0 || p->T > (int64_t)INT32_MAX / 2) return GDN_ERR_UNSUPPORTED;
  if (cu[0] != 0 || cu[p->N] != p->T) return GDN_ERR_INVALID_ARG;
  int64_t all = 0;
  int most = 1;
  plan->bounds = 0;
  for (int d = 0; d < p->N; ++d) {
    if (cu[d + 1] < cu[d]) return GDN_ERR_INVALID_ARG;
    all += chunks_of(cu, d);
    most = std::max(most, chunks_of(cu, d));
    plan->bounds += la_bound(d, cu[d + 1]);
  }
  const double sms = sm_count(), work = (double)all * p->HV;
  plan->len = p->segment > 0 ? std::min(p->segment, most) : most;
  if (p->segment == 0 && most > 1.3 * work / sms && most > 2) {
    auto time = [&](int len, int64_t segments) {
      const double ctas = (double)segments * p->HV, mean = work / ctas;
      if (ctas <= sms) return len + LA_BEGIN;
      if (mean > 0.8 * len) return (double)(int64_t)((ctas + sms - 1) / sms) * (len + LA_BEGIN);
      return (work + LA_BEGIN * ctas) / sms + 0.5 * (len + LA_BEGIN);
    };
    double best = time(most, p->N);
    for (int parts = 2; parts <= most; parts += 1 + parts / 16) {
      const int len = (most + parts - 1) / parts;
      const double t = 1.8 * time(len, segments_of(p, cu, len)) + 4;
      if (t < best) {
        best = t;
        plan->len = len;
      }
    }
  }
  const int64_t total = segments_of(p, cu, plan->len);
  if (total * p->HV > INT32_MAX / 16) return GDN_ERR_UNSUPPORTED;
  plan->total = (int)total;
  plan->split = most > plan->len;
  return GDN_OK;
}

static size_t la_states(const gdn_la_problem* p, const LaPlan& plan) {
  return plan.split ? (size_t)plan.total * p->HV * STATE_F32 * sizeof(float) : 0;
}

// Sums of dq and dk over the value heads of a group, side by side: for each a FP32 tile to a chunk and q/k head (a document's
// chunks begin at t0 / 128 + its number, so that none share one); then for each the counts of heads that are in a tile and a ticket.
static int64_t la_counts(const gdn_la_problem* p) { return p->HV > p->H ? (p->T / LA_CH + p->N + 1) * p->H : 0; }
static size_t la_parts(const gdn_la_problem* p) { return (size_t)la_counts(p) * LA_CH * 128 * sizeof(float); }
static size_t la_sum_bytes(const gdn_la_problem* p) {
  return p->HV > p->H ? 2 * (la_parts(p) + (la_counts(p) + 1) * sizeof(int)) : 0;
}

static bool la_stride(int64_t* s, int heads) {
  if (*s == 0) *s = (int64_t)heads * 128;
  return *s >= (int64_t)heads * 128 && *s % 8 == 0 && *s < (int64_t)1 << 38;
}

// One tensor of a walk: rows of `heads` heads, `token` elements apart.
struct LaTensor {
  const void* base;
  int heads;
  int64_t token;
};

struct LaCall {
  const gdn_la_problem* p;
  LaPlan plan;
  LaWalk w;
  cudaStream_t s;
  bool ok = true;

  LaCall(const gdn_la_problem* prob, const LaPlan& pl, const float* decay, const int32_t* cu, int32_t* err, cudaStream_t st)
      : p(prob), plan(pl), s(st) {
    memset(&w, 0, sizeof w);
    w.seg = {cu, p->N, pl.len, pl.total, p->T, pl.bounds};
    w.decay = decay;
    w.HV = p->HV;
    w.err = err;
  }
  void tensors(const LaTensor& x, const LaTensor& y, const LaTensor& z) {
    auto map = [&](CUtensorMap* m, int* group, const LaTensor& t) {
      *group = p->HV / t.heads;
      if (p->T > 0) ok = ok && make_tmap_strided(m, t.base, p->T, t.heads, t.token, LA_CH);
    };
    map(&w.tx, &w.gx, x);
    map(&w.ty, &w.gy, y);
    map(&w.tz, &w.gz, z);
  }
  void scales(float pairs, float row, float state) {
    w.p_scale = pairs;
    w.row_scale = row;
    w.state_scale = state;
  }
  void check(cudaError_t e) { ok = ok && e == cudaSuccess; }
  // the states that the segments start from, by y and z as set
  void carried(bool reverse, bool exact, const float* init, int init_t, float* sums) {
    if (!ok) return;
    w.sums = sums;
    w.init = nullptr;
    prof_begin(K_LA_SUMS, s);
    check(launch_la_sums(w, reverse, exact, s));
    prof_end(K_LA_SUMS, s);
    const LaCarry c = {w.seg, w.decay, w.HV, init_t, reverse, init, sums, w.err};
    prof_begin(K_LA_CARRY, s);
    check(launch_la_carry(c, s));
    prof_end(K_LA_CARRY, s);
  }
  void start(const float* init, int one_a_segment, int init_t) {
    w.init = init;
    w.init_segments = one_a_segment;
    w.init_t = init_t;
  }
  // to rows of the value heads, `token` elements apart
  void walk(bool reverse, void* out, int64_t token, float* last) {
    w.out = out;
    w.out_token = token;
    w.last = last;
    if (p->T > 0) ok = ok && make_tmap_strided(&w.to, out, p->T, p->HV, token, LA_CH);
    if (!ok) return;
    prof_begin(K_LA_WALK, s);
    check(launch_la_walk(w, reverse, last != nullptr, false, s));
    prof_end(K_LA_WALK, s);
  }
  // to rows of the q/k heads, the sums over their value heads; the first or the second that sums
  void walk_summed(bool reverse, void* out, int64_t token, float* part, int which) {
    if (p->HV == p->H) return walk(reverse, out, token, nullptr);
    w.last = nullptr;
    w.group = p->HV / p->H;
    w.sums = part + which * (la_parts(p) / sizeof(float));
    w.counts = counts(part) + which * (la_counts(p) + 1);
    w.ticket = w.counts + la_counts(p);
    w.out = out;
    w.out_token = token;
    if (p->T > 0) ok = ok && make_tmap_strided(&w.to, out, p->T, p->H, token, LA_CH);
    if (!ok) return;
    prof_begin(K_LA_WALK, s);
    check(launch_la_walk(w, reverse, false, true, s));
    prof_end(K_LA_WALK, s);
  }
  int* counts(float* part) const { return reinterpret_cast<int*>(part + 2 * (la_parts(p) / sizeof(float))); }
};

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_la_workspace_bytes(const gdn_la_problem* p, const int32_t* cu_host, size_t* fwd_bytes, size_t* bwd_bytes) {
  LaPlan plan;
  const gdn_status st = la_plan(p, cu_host, &plan);
  if (st != GDN_OK) return st;
  if (!fwd_bytes || !bwd_bytes) return GDN_ERR_INVALID_ARG;
  *fwd_bytes = la_states(p, plan);
  *bwd_bytes = 2 * la_states(p, plan) + la_sum_bytes(p);
  return GDN_OK;
}

gdn_status gdn_la_fwd(const gdn_la_problem* p, const void* q, const void* k, const void* v, const float* decay,
                      const int32_t* cu_dev, const int32_t* cu_host, const float* s_in, void* o, float* s_out,
                      int32_t* dev_err, void* workspace, size_t ws_bytes, struct CUstream_st* stream) {
  LaPlan plan;
  const gdn_status st = la_plan(p, cu_host, &plan);
  if (st != GDN_OK) return st;
  int64_t qs = p->q_stride, ks = p->k_stride, vs = p->v_stride;
  if (!la_stride(&qs, p->H) || !la_stride(&ks, p->H) || !la_stride(&vs, p->HV)) return GDN_ERR_INVALID_ARG;
  if (!on_words(decay, cu_dev, dev_err) || !decay || !cu_dev || !dev_err) return GDN_ERR_INVALID_ARG;
  if (p->T > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))) return GDN_ERR_INVALID_ARG;
  if ((s_in && !aligned16(s_in)) || (s_out && !aligned16(s_out))) return GDN_ERR_INVALID_ARG;
  if (plan.split && !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
  if (ws_bytes < la_states(p, plan)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (p->T == 0 && !s_out) return GDN_OK;
  LaCall c(p, plan, decay, cu_dev, dev_err, stream);
  c.tensors({q, p->H, qs}, {k, p->H, ks}, {v, p->HV, vs});
  c.scales(p->scale, p->scale, 1.f);
  c.start(s_in, 0, 0);
  if (plan.split) {
    c.carried(false, s_out != nullptr, s_in, 0, static_cast<float*>(workspace));
    c.start(static_cast<float*>(workspace), 1, 0);
  }
  c.walk(false, o, (int64_t)p->HV * 128, s_out);
  return c.ok ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_la_bwd(const gdn_la_problem* p, const void* q, const void* k, const void* v, const float* decay,
                      const int32_t* cu_dev, const int32_t* cu_host, const float* s_in, const void* dO,
                      const float* ds_out, void* dq, void* dk, void* dv, float* ds_in, int32_t* dev_err, void* workspace,
                      size_t ws_bytes, struct CUstream_st* stream) {
  LaPlan plan;
  const gdn_status st = la_plan(p, cu_host, &plan);
  if (st != GDN_OK) return st;
  int64_t qs = p->q_stride, ks = p->k_stride, vs = p->v_stride;
  if (!la_stride(&qs, p->H) || !la_stride(&ks, p->H) || !la_stride(&vs, p->HV)) return GDN_ERR_INVALID_ARG;
  if (!on_words(decay, cu_dev, dev_err) || !decay || !cu_dev || !dev_err) return GDN_ERR_INVALID_ARG;
  if (p->T > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(dq) || !aligned16(dk) ||
                   !aligned16(dv)))
    return GDN_ERR_INVALID_ARG;
  if ((s_in && !aligned16(s_in)) || (ds_out && !aligned16(ds_out)) || (ds_in && !aligned16(ds_in))) return GDN_ERR_INVALID_ARG;
  size_t need_fwd, need;
  gdn_la_workspace_bytes(p, cu_host, &need_fwd, &need);
  if (need && !aligned16(workspace)) return GDN_ERR_INVALID_ARG;
  if (ws_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
  if (p->T == 0 && !ds_in) return GDN_OK;
  const LaTensor tq = {q, p->H, qs}, tk = {k, p->H, ks}, tv = {v, p->HV, vs}, td = {dO, p->HV, (int64_t)p->HV * 128};
  float* states = static_cast<float*>(workspace);
  const size_t values = la_states(p, plan) / sizeof(float);
  float *wstates = states + values, *part = wstates + values;
  LaCall c(p, plan, decay, cu_dev, dev_err, stream);
  const float *w_start = ds_out, *s_start = s_in;
  // The counts of heads and the tickets, zero before the first kernel of this call: a walk that follows another does not wait
  // for it, so nothing it reads may come from there, or from anything but what had ended before that one went on.
  if (p->HV > p->H && p->T > 0) c.check(cudaMemsetAsync(c.counts(part), 0, 2 * (la_counts(p) + 1) * sizeof(int), stream));
  if (plan.split) {   // the states that segments start from
    c.tensors(tk, tq, td);
    c.scales(p->scale, 1.f, p->scale);
    c.carried(true, ds_in != nullptr, ds_out, 0, wstates);
    w_start = wstates;
    if (p->T > 0) {
      c.tensors(td, tv, tk);
      c.scales(p->scale, p->scale, 1.f);
      c.carried(false, false, s_in, 1, states);
      s_start = states;
    }
  }
  // The three walks need nothing of one another, so each begins as the one before runs out of work (8 documents of 8,192 tokens,
  // 48 heads on 16: 1,790 us, one after the other 1,911; a ragged pack of 7 225 and 281); but dk's reads the gradients of the
  // states before dv's writes over them.
  const bool in_place = ds_in && ds_in == ds_out && !plan.split;
  auto dk_walk = [&] {   // by dv's states, seen from the other side
    c.tensors(tv, td, tq);
    c.scales(p->scale, 1.f, p->scale);
    c.start(w_start, plan.split, 1);
    c.walk_summed(true, dk, ks, part, 0);
  };
  auto dv_walk = [&] {   // and the gradients of the states; Z[dk][dv]
    c.tensors(tk, tq, td);
    c.scales(p->scale, 1.f, p->scale);
    c.start(w_start, plan.split, 0);
    c.walk(true, dv, vs, ds_in);
  };
  if (p->T == 0) {
    dv_walk();
    return c.ok ? GDN_OK : GDN_ERR_CUDA;
  }
  if (in_place) {
    dk_walk();
    c.w.leads = 1;
    dv_walk();
  } else {
    c.w.leads = 1;
    dv_walk();
    c.w.leads = 0;
    c.w.follows = 1;
    dk_walk();
  }
  // dq; Z[dv][dk], the state before each chunk
  c.w.leads = 0;
  c.w.follows = 1;
  c.tensors(td, tv, tk);
  c.scales(p->scale, p->scale, 1.f);
  c.start(s_start, plan.split, !plan.split);
  c.walk_summed(false, dq, qs, part, 1);
  return c.ok ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
