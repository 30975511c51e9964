// Eviction from the cache by accumulated attention weight.
//
// Every lane -- (shard i, sequence b, KV head h), n cached tokens -- keeps
// k = min(keep[b, i], n) tokens of the largest mass; the first n_sink and the
// last n_recent positions count as mass +inf, a NaN mass as -inf, and ties go to
// the lower cache index. The kept set is the same whatever the order of the work.
//
// The kept rows end up at local indices [0, k) of their shard. Rows already
// there stay; the kept rows behind (as many as there are holes before k) move
// into the holes, the j-th into the j-th, both ascending. Sources lie at or
// past k and destinations before it, so the copies are in place and
// independent of each other, and they are the fewest possible: about
// k (n - k) / n rows instead of k. No row changes its shard or head.
//
// select_kernel: one CTA per lane finds the k-th largest key (32-bit
// order-preserving integers) by radix selection, three digits of 11, 11 and 10
// bits from the top, over keys kept in shared memory (re-read from L2 where a
// lane has more than it holds). Each warp then takes a contiguous part of the
// lane: it counts its keys above and equal to the threshold, before and behind
// k, one scan over the warps' counts tells every warp which ties it keeps and
// where its holes and sources go, and a last pass lists them. Bound by the
// instructions of these passes (170 a warp and 32 tokens, two thirds of the issue
// slots) and, for short lanes, by their latency, not by the 4 bytes read per
// token: 512 lanes of 2K tokens 15 us, 256 of 16K 31 us (37 with the masses read
// one at a time), 64 of 25K 28 us.
// move_kernel: a warp looks up 32 moves at once, a lane each (list, block
// table, mass, position), and then copies their rows, four 16-byte pieces per
// lane in flight. Bound by HBM: rows are read and written once. Four pieces
// and 40 warps an SM against eight and 16 (registers): half of 32 x 32K tokens
// x 4 heads of 128 in bf16, 1.07 GB moved, 220 us with the selection against
// 366; two pieces and 64 warps 230, four and 64 (spilled) 308. Today 211 us, of
// which the moves are 177: 6.1 TB/s of reads and writes. 8-bit values lie
// transposed in their block, a token's bytes block_size apart: a lane each move
// makes neighbouring tokens' bytes neighbouring lanes' (the same shape in E4M3
// 334 us, 263 with blocks of 64 tokens; a warp a move 612, 1146; 84 us of bytes).
// 4-bit values share words between two tokens, set by atomics: 206 us, 47 of
// bytes; one exclusive-or instead of two atomics 230, plain rewrites of words
// whose other token is known 258.
#include <climits>
#include <mutex>

#include "dcp_mx4.cuh"

namespace dcp {
namespace {

// Keys in shared memory: 100 KB, so that two CTAs of 512 threads fit an SM (the
// form of 1024 threads, for fewer lanes than SMs, has the SM to itself and could
// hold twice as many; not measured).
constexpr int kKeyCache = 25600;
constexpr int kMoveThreads = 256;

struct EvictParams {
  ShardSet sh;
  const int32_t* seq_lens;
  const int32_t* starts;
  const int32_t* keep;
  const float* mass_in;
  const int32_t* pos_in;
  const int32_t* known;
  const int32_t* total;
  float* mass_out;
  int32_t* pos_out;
  int32_t* new_starts;
  int32_t* new_lens;
  int32_t* counts;  // workspace: moves of every lane
  int32_t* lists;   // workspace: holes and sources, in the lane's range of a mass row
  int32_t* err;
  long long cap;
  int B, N, Hkv, Bs;
  int n_sink, n_recent;
  int per;    // move_kernel: CTAs of a lane
  int cache;  // select_kernel: keys in shared memory
};

// Tokens [start, start + n) of shard i of sequence b, n cut to the mass rows.
// A shard that starts before an earlier one (or before 0) holds none, so that
// no two shards share a token.
__device__ __forceinline__ int lane_tokens(const EvictParams& p, int b, int i, int* start) {
  const int32_t* st = p.starts + (size_t)b * p.N;
  const int s = st[i];
  int e = p.seq_lens[b];
  if (i + 1 < p.N) e = min(e, st[i + 1]);
  *start = s;
  int least = 0;
  for (int j = 0; j < i; ++j) least = max(least, st[j]);
  if (s < least) return 0;
  if ((long long)e > p.cap) e = (int)p.cap;
  return max(0, e - s);
}

__device__ __forceinline__ int lane_keep(const EvictParams& p, int b, int i, int n) {
  return min(max(p.keep[(size_t)b * p.N + i], 0), n);
}

struct LaneView {
  const float* mass;
  const int32_t* pos;
  int known, shift, sink, recent;  // position of token t past `known`: t + shift
};

__device__ __forceinline__ int position(const LaneView& v, int t) { return v.pos && t < v.known ? v.pos[t] : t + v.shift; }

// Key of a token by its mass and position; larger: kept earlier.
__device__ __forceinline__ uint32_t sort_key(const LaneView& v, float m, int pos) {
  if (m != m) m = -INFINITY;
  if (pos < v.sink || pos >= v.recent) m = INFINITY;
  if (m == 0.f) m = 0.f;  // one zero
  const uint32_t u = __float_as_uint(m);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// f(t, key) for this thread's tokens t = tid, tid + THREADS, ... below n of the
// lane at `start`, eight loads at a time (f writes to memory, past which the
// compiler moves no load).
template <int THREADS, class F>
__device__ __forceinline__ void each_key(const LaneView& v, int start, int n, int tid, F f) {
  constexpr int kAhead = 8;
  for (int t = tid; t < n; t += THREADS * kAhead) {
    float m[kAhead];
    int pos[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int at = start + min(t + a * THREADS, n - 1);
      m[a] = v.mass[at];
      pos[a] = position(v, at);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (t + a * THREADS < n) f(t + a * THREADS, sort_key(v, m[a], pos[a]));
  }
}

__device__ __forceinline__ int warp_scan(int x) {  // inclusive
  const int lane = threadIdx.x & 31;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kWarps = THREADS / 32, kBins = 2048, kPer = kBins / THREADS;
  extern __shared__ uint32_t keys[];  // p.cache of them
  __shared__ int hist[kBins];
  __shared__ int s_bin, s_left;
  __shared__ int part[kWarps];
  __shared__ int counts[kWarps][4];  // keys above the threshold before and behind k, equal ones likewise
  const int h = blockIdx.x % p.Hkv, u = blockIdx.x / p.Hkv;
  const int i = u % p.N, b = u / p.N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int start;
  const int n = lane_tokens(p, b, i, &start), k = lane_keep(p, b, i, n);
  // where the shard's kept tokens start, and the sequence's new length
  int base = 0, all = 0, least = 0;
  for (int j = 0; j < p.N; ++j) {
    int s;
    const int nj = lane_tokens(p, b, j, &s);
    const int kj = lane_keep(p, b, j, nj);
    if (j < i) base += kj;
    all += kj;
    if (tid == 0 && s < least) raise_flag(p.err, DCP_DEVERR_POSITION);
    least = max(least, s);
  }
  const int len = p.seq_lens[b];
  if (h == 0 && tid == 0) {
    p.new_starts[(size_t)b * p.N + i] = base;
    if (i == 0) p.new_lens[b] = all;
    if ((long long)len > p.cap) raise_flag(p.err, DCP_DEVERR_TABLE_RANGE);
  }
  const size_t row = ((size_t)b * p.Hkv + h) * (size_t)p.cap;
  LaneView v;
  v.mass = p.mass_in + row;
  v.pos = p.pos_in ? p.pos_in + row : nullptr;
  v.known = p.known ? p.known[b] : 0;
  const int total = p.total ? p.total[b] : len;
  v.shift = total - len;
  v.sink = p.n_sink;
  v.recent = total - p.n_recent;
  float* mass_out = p.mass_out + row + base;
  int32_t* pos_out = p.pos_out + row + base;

  if (k == 0 || k == n) {  // none stays, or all do
    for (int t = tid; t < k; t += THREADS) {
      mass_out[t] = v.mass[start + t];
      pos_out[t] = position(v, start + t);
    }
    if (tid == 0) p.counts[blockIdx.x] = 0;
    return;
  }

  // the k-th largest key: `prefix` of its top bits, `left` of the tokens that
  // share them are kept
  const bool cached = n <= p.cache;
  uint32_t prefix = 0;
  int left = k;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int above = shift + (pass == 2 ? 10 : 11);  // bits already fixed lie above
    for (int j = tid; j < kBins; j += THREADS) hist[j] = 0;
    __syncthreads();
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    auto count = [&](uint32_t key) {
      if (pass == 0 || (key >> above) == (prefix >> above)) atomicAdd(&hist[(key >> shift) & mask], 1);
    };
    if (pass == 0 || !cached) {
      each_key<THREADS>(v, start, n, tid, [&](int t, uint32_t key) {
        if (pass == 0 && cached) keys[t] = key;
        count(key);
      });
    } else {
#pragma unroll 4
      for (int t = tid; t < n; t += THREADS) count(keys[t]);
    }
    __syncthreads();
    // the bin where the count from the top reaches `left`: thread t owns the
    // kPer bins from kBins - 1 - t kPer down
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) mine += hist[kBins - 1 - tid * kPer - j];
    const int inc = warp_scan(mine);
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    const int pre = warp_scan(lane < kWarps ? part[lane] : 0);
    int before = inc - mine + (warp > 0 ? __shfl_sync(0xffffffffu, pre, warp - 1) : 0);
    if (before < left && before + mine >= left) {
      for (int j = 0; j < kPer; ++j) {
        const int bin = kBins - 1 - tid * kPer - j, c = hist[bin];
        if (before + c >= left) {
          s_bin = bin;
          s_left = left - before;
          break;
        }
        before += c;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    left = s_left;
  }

  // a warp's part of the lane, in order
  const int seg = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int t0 = min(n, warp * seg), t1 = min(n, t0 + seg);
  {
    int gl = 0, gh = 0, el = 0, eh = 0;
#pragma unroll 4
    for (int t = t0 + lane; t < t1; t += 32) {
      const uint32_t key = cached ? keys[t] : sort_key(v, v.mass[start + t], position(v, start + t));
      gl += key > prefix && t < k;
      gh += key > prefix && t >= k;
      el += key == prefix && t < k;
      eh += key == prefix && t >= k;
    }
    gl = __reduce_add_sync(0xffffffffu, gl);
    gh = __reduce_add_sync(0xffffffffu, gh);
    el = __reduce_add_sync(0xffffffffu, el);
    eh = __reduce_add_sync(0xffffffffu, eh);
    if (lane == 0) {
      counts[warp][0] = gl;
      counts[warp][1] = gh;
      counts[warp][2] = el;
      counts[warp][3] = eh;
    }
  }
  __syncthreads();
  // lane w: warp w's ties that are kept (the first `left` of the lane), its holes and sources
  int ties, hole0, src0, holes;
  {
    int c[4] = {0, 0, 0, 0}, size_low = 0;
    if (lane < kWarps) {
      for (int j = 0; j < 4; ++j) c[j] = counts[lane][j];
      const int a = min(n, lane * seg), e = min(n, a + seg);
      size_low = max(0, min(e, k) - a);  // its tokens before k
    }
    const int eq = c[2] + c[3], eq_before = warp_scan(eq) - eq;
    const int kept = min(max(left - eq_before, 0), eq);
    const int kept_low = min(kept, c[2]);
    const int nh = size_low - c[0] - kept_low, ns = c[1] + kept - kept_low;
    const int h_inc = warp_scan(nh), s_inc = warp_scan(ns);
    ties = __shfl_sync(0xffffffffu, kept, warp);
    hole0 = __shfl_sync(0xffffffffu, h_inc - nh, warp);
    src0 = __shfl_sync(0xffffffffu, s_inc - ns, warp);
    holes = __shfl_sync(0xffffffffu, h_inc, 31);
  }
  int32_t* dst = p.lists + row + start;
  int32_t* src = dst + n / 2;  // holes and sources are equally many, at most n / 2
  const unsigned lower = (1u << lane) - 1;
  constexpr int kAhead = 8;
  for (int t4 = t0; t4 < t1; t4 += 32 * kAhead) {
    float m[kAhead];
    int pos[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int t = t4 + 32 * a + lane;
      const bool wanted = t < t1 && (t < k || !cached);
      m[a] = wanted ? v.mass[start + t] : 0.f;
      pos[a] = wanted ? position(v, start + t) : 0;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int t = t4 + 32 * a + lane;
      const bool in = t < t1;
      const uint32_t key = !in ? 0u : cached ? keys[t] : sort_key(v, m[a], pos[a]);
      const bool eq = in && key == prefix;
      const unsigned eqs = __ballot_sync(0xffffffffu, eq);
      const bool kept = in && (key > prefix || (eq && __popc(eqs & lower) < ties));
      ties = max(0, ties - __popc(eqs));
      const bool hole = in && t < k && !kept, come = kept && t >= k;
      const unsigned hs = __ballot_sync(0xffffffffu, hole), cs = __ballot_sync(0xffffffffu, come);
      if (hole) dst[hole0 + __popc(hs & lower)] = t;
      if (come) src[src0 + __popc(cs & lower)] = t;
      hole0 += __popc(hs);
      src0 += __popc(cs);
      if (kept && t < k) {
        mass_out[t] = m[a];
        pos_out[t] = pos[a];
      }
    }
  }
  if (tid == 0) p.counts[blockIdx.x] = holes;
}

// KV: 0 bf16, 1 E4M3, 2 microscaled 4-bit. D 576: one latent row, no value pool.
template <int KV, int D>
__global__ void __launch_bounds__(kMoveThreads, KV == 1 && D != 576 ? 4 : 5) move_kernel(const __grid_constant__ EvictParams p) {
  constexpr bool kMla = D == 576;
  constexpr int kAhead = 4;  // pieces in flight per lane
  // 16-byte pieces of a key row; bf16 value rows have as many, behind them
  constexpr int kRow = KV == 0 ? D * 2 : KV == 1 ? D : D / 2;
  constexpr int kK = kRow / 16, kPieces = KV == 0 && !kMla ? 2 * kK : kK;
  grid_wait();  // the selection
  const int lid = blockIdx.x / p.per, chunk = blockIdx.x - lid * p.per;
  const int h = lid % p.Hkv, u = lid / p.Hkv;
  const int i = u % p.N, b = u / p.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = p.counts[lid];
  int j0 = (chunk * (kMoveThreads / 32) + warp) * 32;
  if (j0 >= count) return;
  int start;
  const int n = lane_tokens(p, b, i, &start);
  const size_t row = ((size_t)b * p.Hkv + h) * (size_t)p.cap;
  const int32_t* dst = p.lists + row + start;
  const int32_t* src = dst + n / 2;
  const size_t out = row + p.new_starts[(size_t)b * p.N + i];
  LaneView v;
  v.mass = p.mass_in + row;
  v.pos = p.pos_in ? p.pos_in + row : nullptr;
  v.known = p.known ? p.known[b] : 0;
  v.shift = (p.total ? p.total[b] : p.seq_lens[b]) - p.seq_lens[b];
  const int32_t* table = p.sh.table[i] + (size_t)b * p.sh.max_blocks[i];
  unsigned char* kp = static_cast<unsigned char*>(const_cast<void*>(p.sh.k[i]));
  unsigned char* vp = static_cast<unsigned char*>(const_cast<void*>(p.sh.v[i]));

  for (; j0 < count; j0 += p.per * kMoveThreads) {
    // a lane's move: row numbers (of all blocks' rows of this pool) to and from; -1: none
    long long to = -1, from = -1;
    if (j0 + lane < count) {
      const int t = dst[j0 + lane], f = src[j0 + lane];
      p.mass_out[out + t] = v.mass[start + f];
      p.pos_out[out + t] = position(v, start + f);
      const int lt = t / p.Bs, lf = f / p.Bs;
      if (lf >= p.sh.max_blocks[i]) {  // t < f
        raise_flag(p.err, DCP_DEVERR_TABLE_RANGE);
      } else {
        const int pt = table[lt], pf = table[lf];
        if (pt < 0 || pt >= p.sh.nblk[i] || pf < 0 || pf >= p.sh.nblk[i]) {
          raise_flag(p.err, DCP_DEVERR_BLOCK_RANGE);
        } else {
          to = ((long long)pt * p.Hkv + h) * p.Bs + t - lt * p.Bs;
          from = ((long long)pf * p.Hkv + h) * p.Bs + f - lf * p.Bs;
        }
      }
    }
    const int moves = min(32, count - j0);
    // 16-byte pieces of the rows, the moves' pieces laid end to end over the lanes
    for (int x0 = lane; x0 < moves * kPieces + lane; x0 += 32 * kAhead) {
      uint4 piece[kAhead];
      unsigned char* at[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int x = x0 + 32 * a, m = x / kPieces, c = x - m * kPieces;
        const long long t = __shfl_sync(0xffffffffu, to, m & 31), f = __shfl_sync(0xffffffffu, from, m & 31);
        at[a] = nullptr;
        if (x < moves * kPieces && t >= 0) {
          if constexpr (KV == 2) {  // keys of a tile are row by row, its scales behind them
            const unsigned char* s = kp + (f / kMxTile) * mx4_tile_bytes(D) + (f % kMxTile) * kRow + c * 16;
            at[a] = kp + (t / kMxTile) * mx4_tile_bytes(D) + (t % kMxTile) * kRow + c * 16;
            piece[a] = *reinterpret_cast<const uint4*>(s);
          } else {
            unsigned char* pool = c < kK ? kp : vp;
            const int o = (c < kK ? c : c - kK) * 16;
            at[a] = pool + t * kRow + o;
            piece[a] = *reinterpret_cast<const uint4*>(pool + f * kRow + o);
          }
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (at[a]) *reinterpret_cast<uint4*>(at[a]) = piece[a];
    }
    if constexpr (KV == 1 && !kMla) {
      // values: D bytes, a block's tokens apart; a lane each move, whose
      // neighbours' bytes lie beside its own (with few moves, several lanes)
      constexpr int kBytes = 16;  // in flight
      int wide = 32;
      while (wide / 2 >= moves) wide /= 2;
      const long long t = __shfl_sync(0xffffffffu, to, lane & (wide - 1)), f = __shfl_sync(0xffffffffu, from, lane & (wide - 1));
      if (t >= 0) {
        unsigned char* dst8 = vp + (t / p.Bs) * D * p.Bs + t % p.Bs;
        const unsigned char* src8 = vp + (f / p.Bs) * D * p.Bs + f % p.Bs;
#pragma unroll 1
        for (int d = lane / wide * kBytes; d < D; d += 32 / wide * kBytes) {
          unsigned char byte[kBytes];
#pragma unroll
          for (int a = 0; a < kBytes; ++a) byte[a] = src8[(d + a) * p.Bs];
#pragma unroll
          for (int a = 0; a < kBytes; ++a) dst8[(d + a) * p.Bs] = byte[a];
        }
      }
    }
    if constexpr (KV == 2) {
      // scales: D / 32 bytes of either pool, a lane each move
      if (to >= 0) {
        const size_t st = (to / kMxTile) * mx4_tile_bytes(D) + mx4_tile_codes(D) + (to % kMxTile) * (D / 32);
        const size_t sf = (from / kMxTile) * mx4_tile_bytes(D) + mx4_tile_codes(D) + (from % kMxTile) * (D / 32);
        unsigned char k8[D / 32], v8[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) k8[c] = kp[sf + c], v8[c] = vp[sf + c];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) kp[st + c] = k8[c], vp[st + c] = v8[c];
      }
      // values: the row's nibbles of D / 4 words; two moves may share a word
      constexpr int kWords = D / 4, kPer = D / 32;
      for (int x0 = lane; x0 < moves * kWords + lane; x0 += 32 * kAhead) {
        uint32_t word[kAhead];
        unsigned int* at[kAhead];
        int n4[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int x = x0 + 32 * a, m = x / kWords, w = x - m * kWords, gr = w / kPer;
          const long long t = __shfl_sync(0xffffffffu, to, m & 31), f = __shfl_sync(0xffffffffu, from, m & 31);
          at[a] = nullptr;
          if (x < moves * kWords && t >= 0) {
            const int rt = (int)(t % kMxTile), rf = (int)(f % kMxTile);
            auto place = [&](long long r, int s) {
              return vp + (r / kMxTile) * mx4_tile_bytes(D) + (s / 8) * (4 * D) + (gr * 4 + (s % 8) / 2) * (D / 8) + 4 * (w % kPer);
            };
            word[a] = (*reinterpret_cast<const uint32_t*>(place(f, rf)) >> (4 * (rf & 1))) & 0x0F0F0F0Fu;
            at[a] = reinterpret_cast<unsigned int*>(place(t, rt));
            n4[a] = 4 * (rt & 1);
          }
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
          if (at[a]) {
            atomicAnd(at[a], ~(0x0F0F0F0Fu << n4[a]));
            atomicOr(at[a], word[a] << n4[a]);
          }
      }
    }
  }
}

template <int THREADS>
cudaError_t launch_select(EvictParams& p, int lanes, int cache, cudaStream_t st) {
  static std::mutex mu;
  static bool set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !set[dev]) {
      e = cudaFuncSetAttribute(select_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, cache * 4);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) set[dev] = true;
    }
  }
  p.cache = cache;
  select_kernel<THREADS><<<lanes, THREADS, cache * 4, st>>>(p);
  return cudaGetLastError();
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t evict_workspace(const dcp_attn_desc& d, int B, int N, long long cap) {
  return align256(sizeof(int32_t) * (size_t)B * N * d.num_kv_heads) +
         align256(sizeof(int32_t) * (size_t)B * d.num_kv_heads * (size_t)cap);
}

cudaError_t launch_evict(const dcp_attn_desc& d, const ShardSet& sh, int N, const int32_t* seq_lens,
                         const int32_t* starts, int B, const int32_t* keep, int n_sink, int n_recent,
                         const float* mass_in, const int32_t* pos_in, const int32_t* known, const int32_t* total,
                         long long cap, float* mass_out, int32_t* pos_out, int32_t* new_starts, int32_t* new_lens,
                         void* ws, int32_t* err, cudaStream_t st) {
  DeviceInfo di;
  if (device_info(&di) != 0) return cudaErrorUnknown;
  EvictParams p;
  p.sh = sh;
  p.seq_lens = seq_lens;
  p.starts = starts;
  p.keep = keep;
  p.mass_in = mass_in;
  p.pos_in = pos_in;
  p.known = known;
  p.total = total;
  p.mass_out = mass_out;
  p.pos_out = pos_out;
  p.new_starts = new_starts;
  p.new_lens = new_lens;
  p.counts = static_cast<int32_t*>(ws);
  p.lists = reinterpret_cast<int32_t*>(static_cast<char*>(ws) +
                                       align256(sizeof(int32_t) * (size_t)B * N * d.num_kv_heads));
  p.err = err;
  p.cap = cap;
  p.B = B;
  p.N = N;
  p.Hkv = d.num_kv_heads;
  p.Bs = d.block_size;
  p.n_sink = n_sink;
  p.n_recent = n_recent;
  const int lanes = B * N * d.num_kv_heads;
  // Lanes of up to about 4096 tokens (the mean lane of the longest sequence
  // allowed decides) take CTAs of 256 threads, of which eight fit an SM. Longer
  // ones take 512 threads, two to an SM for the keys' sake, or 1024 where the
  // lanes are too few to give every SM two.
  cudaError_t e;
  if (cap / N <= 4096) e = launch_select<256>(p, lanes, 4096, st);
  else if (lanes > di.sm_count) e = launch_select<512>(p, lanes, kKeyCache, st);
  else e = launch_select<1024>(p, lanes, kKeyCache, st);
  if (e != cudaSuccess) return e;
  // enough CTAs to fill the GPU several times over, whatever the lanes; no
  // more than the moves a lane can have (half its tokens) give work
  const long long most = (cap / 2 + kMoveThreads - 1) / kMoveThreads;
  long long per = (di.sm_count * 16 + lanes - 1) / lanes;
  if (per > most) per = most > 0 ? most : 1;
  p.per = (int)per;
  const unsigned grid = (unsigned)(per * lanes);
  const int kv = d.kv_dtype == DCP_KV_BF16 ? 0 : d.kv_dtype == DCP_KV_FP8_E4M3 ? 1 : 2;
  auto kernel = move_kernel<0, 576>;
  if (d.kind == DCP_KIND_MLA) kernel = kv == 0 ? move_kernel<0, 576> : move_kernel<1, 576>;
  else if (d.head_dim_k == 128) kernel = kv == 0 ? move_kernel<0, 128> : kv == 1 ? move_kernel<1, 128> : move_kernel<2, 128>;
  else kernel = kv == 0 ? move_kernel<0, 64> : kv == 1 ? move_kernel<1, 64> : move_kernel<2, 64>;
  return launch_behind(kernel, grid, kMoveThreads, 0, st, p);
}

}  // namespace dcp
