// What the attention-weight kernels share: parameters, the tokens of a lane,
// and a CTA's place in the work.
//
// The tokens of all (shard, sequence, KV head) lanes are laid end to end in
// tiles of 128, each CTA takes an equal run of them and finds its place by a
// scan of the lengths (a few thousand integers from L2), so the lengths stay on
// the device and the call is one launch. A lane counts kMassLaneCost tiles more
// than it has, before its first: loading its query rows and constants takes a
// CTA about as long as two tiles (measured on one shape, for all of them: 16 ragged sequences of up to 8K tokens in 4
// shards, 32 query tokens: 46 us at 1, 40 at 2 and 3, 43 at 5).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dcp_internal.cuh"

namespace dcp {

struct MassParams {
  const __nv_bfloat16* q;
  ShardSet sh;
  const int32_t* seq_lens;
  const int32_t* starts;
  const float* lse;
  const float* mass_in;
  float* mass_out;
  int32_t* err;
  long long cap;  // entries of a mass row
  int B, N, qlen, Hq, Hkv, g, Bs;
  float sl2;      // scale * log2(e) (times the 8-bit cache's key scale)
};

// Many query rows per KV head (dcp_mass_tc.cu).
bool mass_tc_eligible(const dcp_attn_desc& d, int qlen);
cudaError_t launch_mass_tc(const dcp_attn_desc& d, const MassParams& p, int sms, cudaStream_t st);

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMassTile = 128;   // tokens of a CTA's tile
constexpr int kMassLaneCost = 2;

// Tokens [start, start + n) of shard i of sequence b; n is cut to the mass rows.
__device__ __forceinline__ int shard_tokens(const MassParams& p, int u, int* start) {
  const int i = u / p.B, b = u - i * p.B;
  const int s = p.starts[(size_t)b * p.N + i];
  int e = p.seq_lens[b];
  if (i + 1 < p.N) e = min(e, p.starts[(size_t)b * p.N + i + 1]);
  *start = s;
  if (s < 0) return 0;
  if ((long long)e > p.cap) e = (int)p.cap;
  return max(0, e - s);
}

// Tiles of a lane of n tokens, and what it counts for.
__device__ __forceinline__ int lane_tiles(int n) { return (n + kMassTile - 1) / kMassTile; }
__device__ __forceinline__ int lane_weight(int n) { return n > 0 ? lane_tiles(n) + kMassLaneCost : 0; }

// The first tile of this CTA's run: its lane's unit and the tiles before that
// unit; returns the run [*x0, *x1) of the tiles laid end to end.
struct RunPlace {
  long long x0, x1, before;  // before: tiles of the units before `unit`
  int unit;
};
template <int THREADS>
__device__ RunPlace find_run(const MassParams& p, RunPlace* shared) {
  __shared__ long long sums[THREADS / 32];
  const int units = p.B * p.N, per = (units + THREADS - 1) / THREADS;
  const int u0 = threadIdx.x * per, u1 = min(units, u0 + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long mine = 0;
  for (int u = u0; u < u1; ++u) {
    int s;
    mine += (long long)lane_weight(shard_tokens(p, u, &s)) * p.Hkv;
    if (blockIdx.x == 0) {
      const int b = u % p.B;
      if (s < 0) raise_flag(p.err, DCP_DEVERR_POSITION);
      if ((long long)p.seq_lens[b] > p.cap) raise_flag(p.err, DCP_DEVERR_TABLE_RANGE);
    }
  }
  long long inc = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  long long base = 0, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) base += sums[w];
    total += sums[w];
  }
  const long long x0 = total * blockIdx.x / gridDim.x, x1 = total * (blockIdx.x + 1) / gridDim.x;
  long long at = base + inc - mine;
  if (threadIdx.x == 0) {
    shared->x0 = x0;
    shared->x1 = x1;
    shared->unit = units;
    shared->before = total;
  }
  __syncthreads();
  if (x0 >= at && x0 < at + mine) {
    for (int u = u0; u < u1; ++u) {
      int s;
      const long long t = (long long)lane_weight(shard_tokens(p, u, &s)) * p.Hkv;
      if (x0 < at + t) {
        shared->unit = u;
        shared->before = at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  return *shared;
}

// Calls f(u, start, n, kvh, t0, t1, r0) for every part of the CTA's run: tiles
// [t0, t1) of KV head kvh of unit u, once per pass over its query rows (from r0).
// f returns whether to go on.
template <class F>
__device__ __forceinline__ void for_parts(const MassParams& p, const RunPlace& run, int rows_per_pass, F f) {
  const int rows = p.qlen * p.g;
  long long x = run.x0, before = run.before;
  for (int u = run.unit; x < run.x1; ++u) {
    int start;
    const int n = shard_tokens(p, u, &start), weight = lane_weight(n);
    while (x < run.x1 && x < before + (long long)weight * p.Hkv) {
      const int kvh = (int)((x - before) / weight);
      const long long lane = before + (long long)kvh * weight + kMassLaneCost;  // place of its first tile
      const long long end = min(run.x1, lane - kMassLaneCost + weight);
      const int t0 = (int)(max(x, lane) - lane), t1 = (int)(end - lane);
      if (t1 > t0)
        for (int r0 = 0; r0 < rows; r0 += rows_per_pass)
          if (!f(u, start, n, kvh, t0, t1, r0)) return;
      x = end;
    }
    before += (long long)weight * p.Hkv;
  }
}

}  // namespace
}  // namespace dcp
