// gdn_la.cuh -- what the walk kernel, its launches and the host layer of the linear attention share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

constexpr int LA_CH = 128;   // tokens of a chunk

// A bound's part of a sum that tells two tables apart: the bits of (number, bound) mixed by shifts and odd factors
// (splitmix64), so that two tables that differ have the same sum once in 2^64.
__host__ __device__ __forceinline__ uint64_t la_bound(int d, int bound) {
  uint64_t x = ((uint64_t)(uint32_t)d << 32 | (uint32_t)bound) + 0x9e3779b97f4a7c15ull;
  x = (x ^ x >> 30) * 0xbf58476d1ce4e5b9ull;
  x = (x ^ x >> 27) * 0x94d049bb133111ebull;
  return x ^ x >> 31;
}

// How the segments of all documents are numbered: document d has max(1, ceil(chunks / len)) of them, in order.
struct LaSegments {
  const int* cu;   // [N+1] on the device
  int N, len, total;   // chunks of a segment; segments as counted from the host's copy
  int64_t T;
  uint64_t bounds;     // la_bound of the host's cu[1 .. N], summed
};

// One walk: out_r = sum over the tokens c that r sees of p_scale a^|r-c| (x_r . y_c) z_c  +  row_scale a^.. Z^T x_r, with
// the state Z = sum of state_scale a^.. y_c z_c^T of the chunks before (forward) or behind (reverse).
struct LaWalk {
  CUtensorMap tx, ty, tz, to;
  LaSegments seg;
  const float* decay;     // [HV] log decays
  int HV, gx, gy, gz;     // value heads to a head of x, y, z
  float p_scale, row_scale, state_scale;
  const float* init;      // states to start from, FP32 [.][HV][128][128], or null: zero
  int init_segments;      // one a segment (else one a document, which then has one segment)
  int init_t;             // stored [z][y] (else [y][z])
  float* sums;            // [segments][HV][y][z]: what each segment adds, for the carry (walks without output);
                          // [chunks][output heads][32][128 rows][4]: heads' sums (walks that sum)
  float* last;            // [N][HV][y][z]: the state that a document leaves, or null
  void* out;              // BF16 rows of 128, heads side by side
  int64_t out_token;      // elements
  // Walks that sum: over the `group` value heads of an output head
  int group;
  int* counts;            // [chunks][output heads]: heads that have been added; zero before the call's first kernel
  int* ticket;            // numbers the CTAs as they begin; the same
  // Walks that need nothing of one another fill the SMs that the one before leaves: `leads`: the next kernel may begin when
  // all CTAs of this one run, and all before it has ended; `follows`: begins then, and does not end before it.  So a walk
  // that follows reads only what was complete before the one that leads went on, never what that one writes.
  int leads, follows;
  int* err;
};

struct LaCarry {
  LaSegments seg;
  const float* decay;
  int HV, init_t, reverse;
  const float* init;   // [N][HV] or null
  float* sums;         // in: what a segment adds; out: the state it starts from
  int* err;
};

// exact: the state is handed out, and keeps FP32's exactness; else it only goes into BF16 results
cudaError_t launch_la_walk(const LaWalk& a, bool reverse, bool exact, bool sum, cudaStream_t s);
cudaError_t launch_la_sums(const LaWalk& a, bool reverse, bool exact, cudaStream_t s);
cudaError_t launch_la_carry(const LaCarry& a, cudaStream_t s);
}  // namespace gdn
