// Partial decode attention over the microscaled 4-bit cache, GQA form.
//
// A lane is (shard, sequence, group of query tokens, KV head, group of heads);
// the lanes' 16-token tiles are laid end to end and every CTA takes an equal run
// of them, whose place it finds by a scan of the lengths (a few hundred or
// thousand integers from L2; a kernel of its own for that, before this one, took
// 6 us of every call). A lane's 16 rows are query heads of one KV head, of up to
// 16 / g query tokens when a group of g heads leaves room. On m16n8k16 fp16
// MMAs with fp32 accumulators (gr = lane / 4, t4 = lane % 4):
//   S[16 x 16]  = sum over the D / 32 scale blocks b of ksc[t, b] (Q_b . Kcode_b)
//                 (two k-steps per block and 8 tokens; the block's scale is a
//                 factor of the whole dot product over the block, applied in
//                 fp32 to the accumulators)
//   O[16 x D] += P[16 x 16] . (vsc[t, b] Vcode), P as fp16 hi + lo, 22
//                 bits (one term would cost the fp32 outputs 2e-4)
// The codes are the operands' own order in the tile (see the layout), so a
// lane loads its share of 8 tokens with one 128-bit shared load and widens a
// byte to an fp16 pair with one conversion; the 4-bit values are exact in
// fp16. Queries are scaled per row by a power of two into fp16's range: their 8
// bits stay exact down to 2^-17 of the row's largest value, and what is below is
// off by 2^-25 of it, less than fp32's sum over the dims loses beside the
// largest (a second term for it would double the score's MMAs).
//
// A CTA has two warps, each of which owns half the scale blocks, and takes its
// run's tiles in rounds of two per warp. Warp w scores tiles 2 w and 2 w + 1 of
// the round and leaves their P in shared memory as MMA operands; then every
// warp multiplies all the round's P with the values of its own blocks. O is at
// most 32 registers a thread that way instead of 64, and nothing is widened
// twice. On 32 sequences x 32K tokens x 64/4 heads of 128: 197 us with the
// merge (193 before P was held relative to each round, see below); one warp doing
// all of a tile by itself 253, a warp per block, four in a CTA, 202 (each P and
// each line of value codes is read four times).
// The warps exchange the rows' maxima over the round's 64 tokens, and P is held
// relative to them, so that fp16's range serves the round and not the row: a
// row's light tokens (behind a sink, say, 2^-25 of it each) keep their bits. The
// round's P V enters O by one factor per row. O and the sums are in units of
// 2^reference, which rises only with a score 2^40 above it.
//
// A value's scale belongs to one (token, 32 dims), so it can leave neither the
// sum over tokens nor the sum over dims: it multiplies the fp16 codes. Scales
// are kept relative to a reference E of their block (2^(c - E), O in units of
// 2^E), raised to the tile's largest scale when a tile exceeds it. Scales
// within 2^-14 .. 2^1 of the reference (checked four tokens at a time by one
// subtraction) are normal fp16 powers of two, exactly. Any other tile (rare:
// values of neighbouring tokens 2^14 apart) takes bf16 operands, whose range
// holds every scale: codes as bf16 subnormals times 2^126, P as bf16 hi + lo
// (16 bits; a third term for tiles this rare is not worth its registers).
//
// Bound: the tensor pipe and instruction issue together. Per SM quadrant an
// m16n8k16 MMA takes 4.2 ns (8 cycles), and about half of it keeps other
// instructions from issuing (one MMA with four 4-bit conversions: 6.2 ns; the
// conversions alone 4.3; with eight FMAs 6.7; the FMAs alone 4.3). A tile's 48
// MMAs (16 of them for P's low terms) and about 400 other instructions (64
// conversions, 32 scale products, 80 for the keys' scales, 55 for the softmax)
// are 97 ns of an SM that way, where its share of HBM delivers the 2,176 bytes
// in 49 ns. Lanes of at most eight rows (HALF: one query token of up to eight
// heads per KV head, say) put P's low terms into the MMA's upper rows, which are
// empty, and leave the upper rows' scores alone: 32 MMAs, 175 us where 16 rows
// take 197 (32 x 32K tokens, 4 KV heads). More warps change nothing: 193 us at 12
// an SM (168 registers), 203 at 16 (128 registers, two stages), both with P
// relative to the row.
#include <cmath>
#include <mutex>

#include "dcp_mx4.cuh"
#include "dcp_tc_ptx.cuh"

namespace dcp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// P at a round's maximum is 2^kHead: two fp16 terms, which end at 2^-24, then
// hold 22 bits of a weight down to 2^-17 of that maximum, and are off by 2^-39
// of it at most further below.
constexpr float kHead = 14.f;
// A row's reference, the unit of its O and sum, follows when a score is 2^kRise
// above it. (fp32 has room for more; a rise costs a rescale of O.)
constexpr float kRise = 40.f;
// A row that sees nothing: finite, so that differences are numbers or infinite.
constexpr float kNone = -3e38f;

template <int D>
struct Mx4Cfg {
  static constexpr int kBlk = D / kMxBlock;             // scale blocks of a row
  static constexpr int kWarps = 2;
  static constexpr int kOwn = kBlk / kWarps;            // scale blocks of a warp
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kMinCtas = 5;                    // an SM (the registers that come of it leave room for 6)
  static constexpr int kTiles = 2 * kWarps;             // of a round
  static constexpr int kStages = 3;                     // rounds
  static constexpr int kTileBytes = mx4_tile_bytes(D);  // 16 tokens, keys or values
  static constexpr int kStageBytes = 2 * kTiles * kTileBytes;
  static constexpr int kOffP = kStages * kStageBytes;   // the round's P: per tile hi and lo operands of 32 lanes
  static constexpr int kOffQ = kOffP + kTiles * 1024;   // the query rows as operands: 512 bytes a k-step
  static constexpr int kOffF = kOffQ + 16 * D * 2;      // the round's value factors: per tile, scale block and t4
  static constexpr int kOffRed = kOffF + kTiles * kBlk * 32;  // per warp and row: four lanes' maxima, or a sum
  static constexpr int kOffTop = kOffRed + kWarps * 16 * 16;    // per warp and scale block: the largest scale code
  static constexpr int kOffBar = kOffTop + kWarps * kBlk * 4;
  static constexpr int kOffTile = kOffBar + kStages * 8;        // per tile of the round, a byte: 0 none, else its tokens
  static constexpr int kOffAbort = kOffTile + 8;                // (+ 128: scales far apart)
  static constexpr int kSmem = kOffAbort + 8;
};

struct Mx4Params {
  const __nv_bfloat16* q;
  ShardSet sh;
  RangeSpec rs;
  int2* runs;      // per lane with tiles: the first of the runs it is in, their number
  float* tmp_o;    // pieces of lanes that several runs share: rows of run r's
  float* tmp_lse;  // first lane's rest from 2 r, of its last lane's begin from 2 r + 1
  int rows_per_lane;
  float* o_parts;
  float* lses;
  int32_t* err;
  int Bseq;     // sequences
  int ngroups;  // token groups per sequence
  int Hq, Hkv, g, groups, Bs;
  int hpl;      // head rows of one query token: min(g, 16)
  float sl2;    // |scale| * log2(e)
  int negate;   // scale < 0: the queries change their sign instead
};

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same onto zero
__device__ __forceinline__ void mma_f16_first(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// x as hi + lo, packed in pairs for an A fragment
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 hf = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - hf.x, x1 - hf.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  const float2 hf = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x0 - hf.x, x1 - hf.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// 32-bit words: 4 (D = 128), 2 (64) or 1 (32)
template <int D>
__device__ __forceinline__ void load_words(uint32_t addr, uint32_t* w) {
  if constexpr (D == 128)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (D == 64)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(w[0]) : "r"(addr));
}
// scale codes of two neighbouring tokens: a word of D / 32 codes for each
template <int D>
__device__ __forceinline__ void load_scales(uint32_t addr, uint32_t* s) {
  if constexpr (D == 128) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(s[0]), "=r"(s[1]) : "r"(addr));
  } else {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(w) : "r"(addr));
    s[0] = w & 0xFFFFu;
    s[1] = w >> 16;
  }
}
// two fp32 values in one register pair: x * f (+ y)
__device__ __forceinline__ void mul2(float* x, unsigned long long f) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2pack(x[0], x[1])), "l"(f));
  f2unpack(r, x[0], x[1]);
}
__device__ __forceinline__ void fma2(float* y, const float* x, unsigned long long f) {
  f2unpack(ffma2(f2pack(x[0], x[1]), f, f2pack(y[0], y[1])), y[0], y[1]);
}
__device__ __forceinline__ void add2(float* y, const float* x) {
  f2unpack(fadd2(f2pack(y[0], y[1]), f2pack(x[0], x[1])), y[0], y[1]);
}
__device__ __forceinline__ int scale_of(uint32_t word, int b) { return (int)((word >> (8 * b)) & 255u); }
// 2^(code - 127) of code b
__device__ __forceinline__ float scale_value(uint32_t word, int b) {
  return __uint_as_float((b == 3 ? word >> 1 : word << (23 - 8 * b)) & 0x7F800000u);
}

// A lane's start (its queries, constants and first copies) takes a CTA about as
// long as twelve tiles, which it counts for, before the lane's first (measured on
// one shape, for all of them: four query tokens of 16 ragged sequences of up to 8K tokens in 4 shards: 53.6 us
// at 4, 44.7 at 8, 42.6 at 12, 42.9 at 16).
constexpr int kLaneCost = 12;

struct Mx4Run {
  long long tiles;   // of all lanes, with their starts
  long long x0, x1;  // this CTA's
  long long before;  // those of the units before `unit`
  int runs, unit;
};
__device__ __forceinline__ int lane_tiles(int lo, int hi) { return (hi - lo + kMxTile - 1) / kMxTile; }
__device__ __forceinline__ int lane_weight(int lo, int hi) { return hi > lo ? lane_tiles(lo, hi) + kLaneCost : 0; }

// The CTA's run, and the unit that its first tile is in. With little work only
// as many CTAs get a run as there are lane starts and a tile in it.
template <int THREADS>
__device__ __forceinline__ void find_run(const RangeSpec& rs, int lpu, Mx4Run* out, long long* sums) {
  const int units = rs.B * rs.N, per = (units + THREADS - 1) / THREADS;
  const int u0 = min(units, (int)threadIdx.x * per), u1 = min(units, u0 + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long mine = 0;
#pragma unroll 4
  for (int u = u0; u < u1; ++u) {
    int lo, hi, start;
    unit_range(rs, u, &lo, &hi, &start);
    mine += lane_weight(lo, hi);
  }
  mine *= lpu;
  long long upto = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  long long at = upto - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) at += sums[w];
    total += sums[w];
  }
  const long long most = total / (kLaneCost + 1);
  const int runs = (int)min((long long)gridDim.x, max(most, 1ll)), c = blockIdx.x;
  const long long x0 = c < runs ? total * c / runs : total, x1 = c < runs ? total * (c + 1) / runs : total;
  if (x0 >= at && x0 < at + mine) {
    int u = u0;
    for (; u < u1; ++u) {
      int lo, hi, start;
      unit_range(rs, u, &lo, &hi, &start);
      const long long w = (long long)lane_weight(lo, hi) * lpu;
      if (x0 < at + w) break;
      at += w;
    }
    out->unit = u;
    out->before = at;
  }
  if (threadIdx.x == 0) {
    out->tiles = total;
    out->x0 = x0;
    out->x1 = x1;
    out->runs = runs;
  }
  __syncthreads();
}

template <int D, bool HALF>
__global__ void __launch_bounds__(Mx4Cfg<D>::kThreads, Mx4Cfg<D>::kMinCtas)
    gqa_mx4_kernel(const __grid_constant__ Mx4Params p) {
  using C = Mx4Cfg<D>;
  constexpr int kBlk = C::kBlk, kOwn = C::kOwn;
  constexpr int kCodes = mx4_tile_codes(D);
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, t4 = lane & 3;
  const uint32_t ring = saddr(smem), pbuf = saddr(smem + C::kOffP) + lane * 16, qfrag = saddr(smem + C::kOffQ) + lane * 16;
  const uint32_t bars = saddr(smem + C::kOffBar);
  float* red = reinterpret_cast<float*>(smem + C::kOffRed);
  const uint32_t factors = saddr(smem + C::kOffF);  // of tile j, t4, block c: + ((4 j + t4) kBlk + c) 8
  int* tops = reinterpret_cast<int*>(smem + C::kOffTop);
  unsigned char* tile_info = smem + C::kOffTile;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < C::kStages; ++i) bar_init(bars + 8 * i, C::kWarps);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  grid_ready();
  __shared__ Mx4Run run;
  __shared__ long long sums[C::kWarps];
  const int lpu = p.Hkv * p.groups;
  find_run<C::kThreads>(p.rs, lpu, &run, sums);
  uint32_t seq = 0;    // rounds of the lanes before: round seq + i of the CTA uses stage (seq + i) % kStages
  bool dead = false;   // a wait gave up: what is left of the run only records its lanes' runs

  long long x = run.x0, before = run.before;
  for (int u = run.unit; x < run.x1;) {
    int lo, hi, start;
    unit_range(p.rs, u, &lo, &hi, &start);
    const int lane_n = lane_tiles(lo, hi), weight = lane_weight(lo, hi);
    if (x >= before + (long long)weight * lpu) {  // the next unit
      before += (long long)weight * lpu;
      ++u;
      continue;
    }
    const int jl = (int)((x - before) / weight);
    const long long first = before + (long long)jl * weight + kLaneCost;  // place of the lane's first tile
    const long long end = min(run.x1, first + lane_n);
    const int t0 = (int)(max(x, first) - first), n_tiles = (int)(end - first) - t0;
    x = end;
    if (end <= first) continue;  // the run ends within the lane's start
    int out_row = -1;            // the lane's own output rows, or those of a piece
    {
      const int c0 = cta_of(first, run.tiles, run.runs), pieces = cta_of(first + lane_n - 1, run.tiles, run.runs) - c0 + 1;
      if (t0 == 0 && threadIdx.x == 0) p.runs[(size_t)u * lpu + jl] = make_int2(c0, pieces);
      if (pieces > 1) out_row = 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
    }
    if (dead) continue;
    const int kvh = jl / p.groups, hg = jl - kvh * p.groups;
    const int shard = u / p.rs.B, rg = u - shard * p.rs.B;
    const int b = rg / p.ngroups, tok0 = (rg - b * p.ngroups) * p.rs.tpr;
    const int head0 = kvh * p.g + hg * 16;
    const int nheads = min(16, p.g - hg * 16);
    const int n_rounds = (n_tiles + C::kTiles - 1) / C::kTiles;
    const int local0 = lo - start + t0 * kMxTile;  // a multiple of 16: lanes start with their shard

    // The places (in tiles of the pool; -1: none) of this warp's tiles 2 warp
    // and 2 warp + 1 of 16 rounds, each window loaded one window ahead.
    const int32_t* table = p.sh.table[shard] + (size_t)b * p.sh.max_blocks[shard];
    auto place = [&](int round0) -> int {
      const int i = (round0 + (lane >> 1)) * C::kTiles + 2 * warp + (lane & 1);
      if (i >= n_tiles) return -1;
      const int lp = local0 + i * kMxTile, lb = lp / p.Bs;
      if (lb >= p.sh.max_blocks[shard]) {
        raise_flag(p.err, DCP_DEVERR_TABLE_RANGE);
        return -1;
      }
      const int phys = table[lb];
      if (phys < 0 || phys >= p.sh.nblk[shard]) {
        raise_flag(p.err, DCP_DEVERR_BLOCK_RANGE);
        return -1;
      }
      return (phys * p.Hkv + kvh) * (p.Bs / kMxTile) + (lp - lb * p.Bs) / kMxTile;
    };
    int win = place(0), win_next = place(16);
    unsigned copied = 0;  // two bits a stage: which of this warp's tiles are there
    const unsigned char* kpool = static_cast<const unsigned char*>(p.sh.k[shard]);
    const unsigned char* vpool = static_cast<const unsigned char*>(p.sh.v[shard]);
    // copy this warp's tiles of round i into their stage (called for i = 0, 1, ... by the whole warp)
    auto issue = [&](int i) {
      if ((i & 15) == 0 && i > 0) {
        win = win_next;
        win_next = place(i + 16);
      }
      const int p0 = __shfl_sync(0xffffffffu, win, (2 * i) & 31), p1 = __shfl_sync(0xffffffffu, win, (2 * i + 1) & 31);
      const uint32_t st = (seq + i) % C::kStages;
      copied = (copied & ~(3u << (2 * st))) | ((p0 >= 0 ? 1u : 0u) | (p1 >= 0 ? 2u : 0u)) << (2 * st);
      if (lane == 0) {
        const uint32_t bar = bars + 8 * st;
        const uint32_t dst = ring + st * C::kStageBytes + 4 * warp * C::kTileBytes;  // K, V of tile 2 warp, then 2 warp + 1
        bar_arrive_tx(bar, ((p0 >= 0 ? 2 : 0) + (p1 >= 0 ? 2 : 0)) * C::kTileBytes);
        if (p0 >= 0) {
          bulk_load(dst, kpool + (size_t)p0 * C::kTileBytes, C::kTileBytes, bar);
          bulk_load(dst + C::kTileBytes, vpool + (size_t)p0 * C::kTileBytes, C::kTileBytes, bar);
        }
        if (p1 >= 0) {
          bulk_load(dst + 2 * C::kTileBytes, kpool + (size_t)p1 * C::kTileBytes, C::kTileBytes, bar);
          bulk_load(dst + 3 * C::kTileBytes, vpool + (size_t)p1 * C::kTileBytes, C::kTileBytes, bar);
        }
      }
    };
    __syncwarp();
    for (int i = 0; i < C::kStages; ++i)
      if (i < n_rounds) issue(i);

    // this lane's rows gr and gr + 8: query row (-1: none; it runs along with zeros), causal limit
    auto query_row = [&](int e) -> long long {
      const int r = gr + 8 * e, js = r / p.hpl, hr = r - js * p.hpl;
      if (js >= p.rs.tpr || tok0 + js >= p.rs.qlen || hr >= nheads) return -1;
      return ((long long)b * p.rs.qlen + tok0 + js) * p.Hq + head0 + hr;
    };
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int jt = tok0 + (gr + 8 * e) / p.hpl;
      lim[e] = p.rs.qlen == 1 || query_row(e) < 0 ? hi : min(hi, p.rs.seq_lens[b] - (p.rs.qlen - 1 - jt));
    }

    // query fragments: the lane's dims of k-step (block, s) are 32 block + 8 t4 + 4 s .. + 3;
    // every row is scaled by a power of two so that its largest value is in
    // [1, 2). Every warp looks at whole rows and lays out its own blocks.
    float rsl2[2];
    {
      uint32_t qa[2 * kOwn][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const long long qr = query_row(e);
        uint4 own[kOwn];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kBlk; ++c) {
          const uint4 raw = qr >= 0 ? *reinterpret_cast<const uint4*>(p.q + qr * D + 32 * c + 8 * t4) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
          if (c / kOwn == warp) own[c % kOwn] = raw;
        }
        top = max(top & 0xFFFFu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int f = min(max((int)(top >> 7), 1), 253);  // exponent field of the largest
        float down = __uint_as_float((uint32_t)(254 - f) << 23);
        if (p.negate) down = -down;
        rsl2[e] = p.sl2 * __uint_as_float((uint32_t)f << 23);
#pragma unroll
        for (int i = 0; i < 4 * kOwn; ++i) {
          const uint32_t w = i % 4 == 0 ? own[i / 4].x : i % 4 == 1 ? own[i / 4].y : i % 4 == 2 ? own[i / 4].z : own[i / 4].w;
          const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
          const __half2 h = __floats2half2_rn(v.x * down, v.y * down);
          qa[i / 2][(i & 1) * 2 + e] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * kOwn; ++i) st_shared_v4(qfrag + 512 * (2 * kOwn * warp + i), qa[i][0], qa[i][1], qa[i][2], qa[i][3]);
    }
    __syncthreads();

    constexpr int kO = HALF ? 2 : 4;
    float o[4 * kOwn][kO];  // rows gr, gr + 8 and dims 32 kOwn warp + 8 m + 2 t4, + 1
#pragma unroll
    for (int m = 0; m < 4 * kOwn; ++m)
#pragma unroll
      for (int e = 0; e < kO; ++e) o[m][e] = 0.f;
    // the rows' references in log2 units and the sums of this lane's columns
    // (bar0: where ref0 rises, before the scale; 175 us instead of 177 for eight
    // rows, but 202 instead of 197 for 16, whose registers are all taken)
    float bar0 = kNone, ref0 = kNone, ref1 = kNone, l[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    // scale code of O's unit: of this warp's blocks, and of block gr % kBlk,
    // whose factors the lane makes; 15 or more, so that the codes within 14
    // below a unit are not negative
    int unit[kOwn], unit_gr = 15;
#pragma unroll
    for (int q = 0; q < kOwn; ++q) unit[q] = 15;
    const int blk = gr % kBlk;
    const uint32_t pick = blk | ((4 + blk) << 4);
    int stopped = -1;  // the round in which a wait gave up

    for (int i = 0; i < n_rounds; ++i) {
      const uint32_t st = (seq + i) % C::kStages, parity = ((seq + i) / C::kStages) & 1u;
      {  // bounded; a warp that gives up takes part in the round's first barrier like the others
        bool landed = false;
        for (uint32_t t = 0; t < kSpinLimit && !landed; ++t) {
          landed = bar_try(bars + 8 * st, parity);
          if ((t & 63u) == 63u && *abort_flag) break;
        }
        if (!landed && !*abort_flag) {
          *abort_flag = 1;
          raise_flag(p.err, DCP_DEVERR_TIMEOUT);
        }
      }
      __syncwarp();
      const int g0 = lo + (t0 + i * C::kTiles) * kMxTile;  // the round's first token
      const uint32_t base = ring + st * C::kStageBytes;
      // S of this warp's tiles: scale-block sums of the codes, times the tokens' scales
      float s[2][2][4];
      const int w0 = g0 + 2 * warp * kMxTile;  // their first token
      const unsigned mine = copied >> (2 * st);
      const int n0 = mine & 1 ? min(kMxTile, hi - w0) : 0, n1 = mine & 2 ? min(kMxTile, hi - w0 - kMxTile) : 0;
      const bool whole = __all_sync(0xffffffffu, n0 + n1 == 2 * kMxTile && min(lim[0], lim[1]) >= w0 + 2 * kMxTile);
      // column 2 t4 + (e & 1) of half h of the warp's tile j is in row e / 2's sight
      auto sees = [&](int j, int h, int e) {
        const int t = 8 * h + 2 * t4 + (e & 1);
        return t < (j ? n1 : n0) && w0 + 16 * j + t < lim[e >> 1];
      };
      if (n0 + n1 > 0) {
        const uint32_t kb = base + 4 * warp * C::kTileBytes;
        uint32_t w[2][2][kBlk], sc[2][2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = kb + 2 * j * C::kTileBytes;
            load_words<D>(at + (8 * h + gr) * (D / 2) + t4 * (D / 8), w[j][h]);
            load_scales<D>(at + kCodes + (8 * h + 2 * t4) * kBlk, sc[j][h]);
          }
#pragma unroll
        for (int c = 0; c < kBlk; ++c) {
          uint32_t q0[4], q1[4];
          load_words<128>(qfrag + 1024 * c, q0);
          load_words<128>(qfrag + 1024 * c + 512, q1);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t b0, b1, b2, b3;
              e2m1x8_to_f16(w[j][h][c], b0, b1, b2, b3);
              float acc[4];
              mma_f16_first(acc, q0, b0, b1);
              mma_f16(acc, q1, b2, b3);
              const unsigned long long f = f2pack(scale_value(sc[j][h][0], c), scale_value(sc[j][h][1], c));
              if (c == 0) {
                mul2(acc, f);
                if (!HALF) mul2(acc + 2, f);
#pragma unroll
                for (int e = 0; e < (HALF ? 2 : 4); ++e) s[j][h][e] = acc[e];
              } else {
                fma2(s[j][h], acc, f);
                if (!HALF) fma2(s[j][h] + 2, acc + 2, f);
              }
            }
        }
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
      if (whole) {
        mx0 = max3f(max3f(s[0][0][0], s[0][0][1], s[0][1][0]), s[0][1][1], max3f(s[1][0][0], s[1][0][1], s[1][1][0]));
        mx0 = fmaxf(mx0, s[1][1][1]);
        if (!HALF) {
          mx1 = max3f(max3f(s[0][0][2], s[0][0][3], s[0][1][2]), s[0][1][3], max3f(s[1][0][2], s[1][0][3], s[1][1][2]));
          mx1 = fmaxf(mx1, s[1][1][3]);
        }
      } else if (n0 + n1 > 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < (HALF ? 2 : 4); ++e)
              if (sees(j, h, e)) {
                if (e < 2) mx0 = fmaxf(mx0, s[j][h][e]);
                else mx1 = fmaxf(mx1, s[j][h][e]);
              }
      }
      // each lane's part of the maxima, for both warps (no shuffles before the
      // barrier); -inf: none of the tokens is in the row's sight
      red[(warp * 16 + gr) * 4 + t4] = mx0;
      if (!HALF) red[(warp * 16 + gr + 8) * 4 + t4] = mx1;
      // Value scales of block gr % kBlk, tokens 2 t4 and 2 t4 + 1 of either half:
      // bytes of z. Less (unit - 14) they are the factors' exponents, near if all
      // within 0 .. 15: 4 (x + 1) as a half's upper byte has the exponent field
      // x + 1. A byte below its bound borrows from the next, but shows itself: it
      // is at least 256 - 238. Tokens that are not there count as near, factor 0.
      uint32_t z[2], there[2], far = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = j ? n1 : n0;
        const uint32_t at = base + (2 * (2 * warp + j) + 1) * C::kTileBytes + kCodes + 2 * t4 * kBlk;
        uint32_t s0[2], s1[2];
        load_scales<D>(at, s0);
        load_scales<D>(at + 8 * kBlk, s1);
        z[j] = __byte_perm(__byte_perm(s0[0], s0[1], pick), __byte_perm(s1[0], s1[1], pick), 0x5410);
        there[j] = ~0u;
        if (n < kMxTile) {
          there[j] = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * (e >> 1) + 2 * t4 + (e & 1) < n) there[j] |= 0xFFu << (8 * e);
          z[j] &= there[j];
        }
        far |= (z[j] - ((uint32_t)(unit_gr - 14) * 0x01010101u & there[j])) & 0xF0F0F0F0u;
      }
      // every warp has left the round before (its P, factors and stage are free),
      // and knows whether a score is too high or a scale far from its unit
      const bool risen = HALF ? mx0 > bar0 : mx0 * rsl2[0] > ref0 + kRise || mx1 * rsl2[1] > ref1 + kRise;
      const bool high = __syncthreads_or(risen || far != 0u);
      if (*abort_flag) {  // (raised before the barrier: the same for all)
        stopped = i;
        break;
      }
      if (i > 0 && i + C::kStages - 1 < n_rounds) issue(i + C::kStages - 1);
      // the rows' maxima in this round, as they were summed and in log2 units
      float s0 = kNone, s1 = kNone;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float4 a = *reinterpret_cast<const float4*>(red + (w * 16 + gr) * 4);
        s0 = max3f(max3f(s0, a.x, a.y), a.z, a.w);
        if (!HALF) {
          const float4 c = *reinterpret_cast<const float4*>(red + (w * 16 + gr + 8) * 4);
          s1 = max3f(max3f(s1, c.x, c.y), c.z, c.w);
        }
      }
      const float x0 = s0 * rsl2[0], x1 = HALF ? x0 : s1 * rsl2[1];
      if (high) {
        int top = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, scale_of(z[j], e));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (t4 == 0 && gr < kBlk) tops[warp * kBlk + gr] = top;
        __syncthreads();
        // the units rise to the round's largest scales
        float down[kOwn];
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
          const int old = unit[q];
#pragma unroll
          for (int w = 0; w < C::kWarps; ++w) unit[q] = max(unit[q], tops[w * kBlk + kOwn * warp + q]);
          const int fall = 127 + old - unit[q];  // 2^(old - new), 0 below 2^-126
          down[q] = fall > 0 ? __uint_as_float((uint32_t)fall << 23) : 0.f;
        }
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) unit_gr = max(unit_gr, tops[w * kBlk + blk]);
        const float top0 = fmaxf(ref0, x0), top1 = fmaxf(ref1, x1);
        const float a0 = ex2_ftz(ref0 - top0), a1 = ex2_ftz(ref1 - top1);
        ref0 = top0;
        ref1 = top1;
        if (HALF) bar0 = (ref0 + kRise) / rsl2[0];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[0][e] *= a0;
          l[1][e] *= a1;
        }
#pragma unroll
        for (int m = 0; m < 4 * kOwn; ++m) {
#pragma unroll
          for (int e = 0; e < kO; ++e) o[m][e] *= (e < 2 ? a0 : a1) * down[m / 4];
        }
      }
      // the factors of this warp's tiles, all blocks
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t x = z[j] - ((uint32_t)(unit_gr - 14) * 0x01010101u & there[j]);
        uint32_t y = (x * 4u + 0x04040404u) & there[j];
        bool apart = false;
        if (high) {  // scales that stay far below their unit, blocks of zeros (scale code 1) aside
          bool low = false;
          y = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int code = scale_of(z[j], e), d = code - unit_gr;
            if (!((there[j] >> (8 * e)) & 1u)) continue;
            if (d >= -14) y |= (uint32_t)(4 * (d + 15)) << (8 * e);
            else low = low || code > 1;
          }
          apart = __any_sync(0xffffffffu, low);
        }
        if (gr < kBlk)
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};\n" ::"r"(factors + ((4 * (2 * warp + j) + t4) * kBlk + gr) * 8),
                       "r"(__byte_perm(y, 0u, 0x1404)), "r"(__byte_perm(y, 0u, 0x3424))
                       : "memory");
        const int n = j ? n1 : n0;
        if (lane == 0) tile_info[2 * warp + j] = (unsigned char)(n <= 0 ? 0 : n | (apart ? 128 : 0));
      }
      // P of this warp's tiles, 2^kHead at the round's maximum; in O's units that
      // is size0, size1 times as much (a row that sees nothing here has P 0, and x
      // anywhere: the factor stays finite)
      const float size0 = ex2_ftz(fminf(x0 - ref0, 100.f) - kHead), size1 = ex2_ftz(fminf(x1 - ref1, 100.f) - kHead);
      if (n0 + n1 > 0) {
        float sum0[2] = {0.f, 0.f}, sum1[2] = {0.f, 0.f};
        const unsigned long long f0 = f2pack(rsl2[0], rsl2[0]), f1 = f2pack(rsl2[1], rsl2[1]);
        const float below[4] = {-s0, -s0, -s1, -s1}, head[2] = {kHead, kHead};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t pa[4], pl[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // (the difference first, which is exact near the maximum: P does not
            // leave fp16, however large the scores)
            float z[4] = {head[0], head[1], head[0], head[1]};
            add2(s[j][h], below);
            fma2(z, s[j][h], f0);
            if (!HALF) {
              add2(s[j][h] + 2, below + 2);
              fma2(z + 2, s[j][h] + 2, f1);
            }
#pragma unroll
            for (int e = 0; e < (HALF ? 2 : 4); ++e) z[e] = ex2_ftz(z[e]);
            if (!whole) {
#pragma unroll
              for (int e = 0; e < (HALF ? 2 : 4); ++e) z[e] = sees(j, h, e) ? z[e] : 0.f;
            }
            add2(sum0, z);
            if constexpr (HALF) {
              split_f16(z[0], z[1], pa[2 * h], pa[2 * h + 1]);
            } else {
              add2(sum1, z + 2);
              split_f16(z[0], z[1], pa[2 * h], pl[2 * h]);
              split_f16(z[2], z[3], pa[2 * h + 1], pl[2 * h + 1]);
            }
          }
          st_shared_v4(pbuf + (2 * warp + j) * 1024, pa[0], pa[1], pa[2], pa[3]);
          if (!HALF) st_shared_v4(pbuf + (2 * warp + j) * 1024 + 512, pl[0], pl[1], pl[2], pl[3]);
        }
        fma2(l[0], sum0, f2pack(size0, size0));
        if (!HALF) fma2(l[1], sum1, f2pack(size1, size1));
      }
      __syncthreads();  // the round's P and factors are there
      // the round's P V on accumulators of its own, added to O once: the MMA's
      // additions truncate, and a run makes many of them
      float acc[4 * kOwn][4];
      auto words = [&](int j, int h, uint32_t* w) {  // codes of tile j, half h, this warp's blocks
        load_words<32 * kOwn>(base + (2 * j + 1) * C::kTileBytes + h * 4 * D + lane * (D / 8) + 4 * kOwn * warp, w);
      };
      auto values = [&](int j, uint32_t (&v)[2][4 * kOwn]) {
        uint32_t f[2 * kOwn];  // block by block, of either half
        load_words<64 * kOwn>(factors + ((4 * j + t4) * kBlk + kOwn * warp) * 8, f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[kOwn];
          words(j, h, w);
#pragma unroll
          for (int q = 0; q < kOwn; ++q) {
            e2m1x8_to_f16(w[q], v[h][4 * q], v[h][4 * q + 1], v[h][4 * q + 2], v[h][4 * q + 3]);
#pragma unroll
            for (int m = 0; m < 4; ++m) v[h][4 * q + m] = mul_f16x2(v[h][4 * q + m], f[2 * q + h]);
          }
        }
      };
      // a byte per tile: all there, and none with scales far apart?
      static_assert(C::kTiles == 4, "a word of tile bytes");
      const uint32_t info = *reinterpret_cast<const volatile uint32_t*>(tile_info);
      const bool all = !((info - 0x01010101u) & 0x80808080u) && !(info & 0x80808080u);
      if (all) {
#pragma unroll
        for (int j = 0; j < C::kTiles; ++j) {
          uint32_t pa[4], pl[4], v[2][4 * kOwn];
          load_words<128>(pbuf + j * 1024, pa);
          if (!HALF) load_words<128>(pbuf + j * 1024 + 512, pl);
          values(j, v);
#pragma unroll
          for (int m = 0; m < 4 * kOwn; ++m) {
            if (j == 0) mma_f16_first(acc[m], HALF ? pa : pl, v[0][m], v[1][m]);
            else mma_f16(acc[m], HALF ? pa : pl, v[0][m], v[1][m]);
          }
          if (!HALF) {
#pragma unroll
            for (int m = 0; m < 4 * kOwn; ++m) mma_f16(acc[m], pa, v[0][m], v[1][m]);
          }
        }
      } else {
#pragma unroll
        for (int m = 0; m < 4 * kOwn; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
#pragma unroll 1
        for (int j = 0; j < C::kTiles; ++j) {
          const int about = (int)(info >> (8 * j)) & 255, n = about & 127;
          if (n == 0) continue;
          uint32_t pa[4], pl[4], v[2][4 * kOwn];
          load_words<128>(pbuf + j * 1024, pa);
          if (!HALF) load_words<128>(pbuf + j * 1024 + 512, pl);
          if (about < 128) {
            values(j, v);
            if (!HALF) {
#pragma unroll
              for (int m = 0; m < 4 * kOwn; ++m) mma_f16(acc[m], pl, v[0][m], v[1][m]);
            }
#pragma unroll
            for (int m = 0; m < 4 * kOwn; ++m) mma_f16(acc[m], pa, v[0][m], v[1][m]);
          } else {
            const uint32_t vt = base + (2 * j + 1) * C::kTileBytes;
#pragma unroll
            for (int q = 0; q < (HALF ? 2 : 4); ++q) {  // P as bf16 hi + lo
              uint32_t &high = HALF ? pa[2 * q] : pa[q], &low = HALF ? pa[2 * q + 1] : pl[q];
              const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&high));
              const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&low));
              split_bf16(hi.x + lo.x, hi.y + lo.y, high, low);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t sc[2], w[kOwn];
              load_scales<D>(vt + kCodes + (8 * h + 2 * t4) * kBlk, sc);
              words(j, h, w);
#pragma unroll
              for (int q = 0; q < kOwn; ++q) {
                uint32_t f = 0u;  // 2^126 times the scales relative to the unit
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int d = 253 + scale_of(sc[e], kOwn * warp + q) - unit[q];
                  if (8 * h + 2 * t4 + e < n && d > 0) f |= (uint32_t)d << (7 + 16 * e);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                  const uint32_t n2 = w[q] >> (8 * m);  // low nibble: token 2 t4, high: 2 t4 + 1
                  const uint32_t raw = ((n2 & 0x7u) << 6) | ((n2 & 0x8u) << 12) | ((n2 & 0x70u) << 18) | ((n2 & 0x80u) << 24);
                  v[h][4 * q + m] = mul_bf16x2(raw, f);
                }
              }
            }
#pragma unroll
            for (int m = 0; m < 4 * kOwn; ++m) {
              if (!HALF) mma_bf16(acc[m], pl, v[0][m], v[1][m]);
              mma_bf16(acc[m], pa, v[0][m], v[1][m]);
            }
          }
        }
      }
      const unsigned long long by0 = f2pack(size0, size0), by1 = f2pack(size1, size1);
#pragma unroll
      for (int m = 0; m < 4 * kOwn; ++m) {
        if constexpr (HALF) add2(acc[m], acc[m] + 2);  // P's low terms
        fma2(o[m], acc[m], by0);
        if constexpr (!HALF) fma2(o[m] + 2, acc[m] + 2, by1);
      }
    }
    if (stopped >= 0) {  // copies in flight must land before the CTA may leave
      const int issued = min(n_rounds, stopped + (stopped > 0 ? C::kStages - 1 : C::kStages));
      if (threadIdx.x == 0)
        for (int r = stopped; r < issued; ++r)
          drain_bar(bars + 8 * ((seq + r) % C::kStages), ((seq + r) / C::kStages) & 1u);
      __syncthreads();
      dead = true;
      continue;
    }
    seq += n_rounds;

    // the rows' sums over lanes and warps
    float l0 = l[0][0] + l[0][1], l1 = l[1][0] + l[1][1];
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    __syncthreads();  // (the exchange of maxima is over, and so are the last round's reads)
    if (t4 == 0) {
      red[warp * 16 + gr] = l0;
      red[warp * 16 + gr + 8] = l1;
    }
    __syncthreads();
    // row (js, hr) of the item: workspace row js * hpl + hr, or output row
    // (query token tok0 + js, head head0 + hr)
#pragma unroll
    for (int e = 0; e < (HALF ? 1 : 2); ++e) {
      const long long qr = query_row(e);
      if (qr < 0) continue;
      float den = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) den += red[w * 16 + gr + 8 * e];
      const size_t row = out_row >= 0 ? (size_t)out_row * p.rows_per_lane + gr + 8 * e
                                         : (size_t)shard * p.Bseq * p.rs.qlen * p.Hq + (size_t)qr;
      float* out = (out_row >= 0 ? p.tmp_o : p.o_parts) + row * D + 32 * kOwn * warp + 2 * t4;
      const float inv = den == 0.f ? 0.f : 1.f / den;  // (NaN stays NaN)
#pragma unroll
      for (int m = 0; m < 4 * kOwn; ++m) {
        const float size = __uint_as_float((uint32_t)unit[m / 4] << 23);
        *reinterpret_cast<float2*>(out + 8 * m) = make_float2(o[m][2 * e] * inv * size, o[m][2 * e + 1] * inv * size);
      }
      if (t4 == 0 && warp == 0)
        (out_row >= 0 ? p.tmp_lse : p.lses)[row] = den == 0.f ? -INFINITY : ((e ? ref1 : ref0) + log2f(den)) * kLn2;
    }
  }
}

// Every output row (sequence, query token, head) merges its pieces -- a
// shard's partial row where one run covered its lane, its runs' rows in the
// workspace otherwise -- by the LSE reweighting. One warp a row; its lanes take
// a piece each to find and weigh the pieces (32 at a time, rescaling what came
// before), then D / 32 columns each. SHARDS: a warp per row of every shard's
// partial result, which merges that shard's pieces only; a row whose lane one
// run covered is there already.
template <int D, bool SHARDS>
__global__ void __launch_bounds__(128) mx4_merge_kernel(const int2* __restrict__ runs,
                                                        const float* __restrict__ tmp_o,
                                                        const float* __restrict__ tmp_lse, int rows_per_lane,
                                                        RangeSpec rs, int Hq, int Hkv, const float* o_parts,
                                                        const float* lses, float* o, float* lse_out) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const long long rd = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);  // the row that is written
  const int G = (rs.qlen + rs.tpr - 1) / rs.tpr, g = Hq / Hkv, groups = (g + 15) / 16;
  const long long rows = (long long)(rs.B / G) * rs.qlen * Hq;
  if (rd >= (SHARDS ? rs.N * rows : rows)) return;
  const long long ro = SHARDS ? rd % rows : rd;
  const int h = (int)(ro % Hq);
  const long long t = ro / Hq;
  const int b = (int)(t / rs.qlen), jt = (int)(t - (long long)b * rs.qlen);
  const int rg = b * G + jt / rs.tpr, js = jt % rs.tpr;
  const int kvh = h / g, hg = (h - kvh * g) / 16;
  const int R = js * (rows_per_lane / rs.tpr) + h - kvh * g - hg * 16;
  const bool mine = SHARDS ? lane == (int)(rd / rows) : lane < rs.N;  // this lane's shard takes part
  bool some = false;
  if (mine) {
    int lo, hi, start;
    unit_range(rs, lane * rs.B + rg, &lo, &hi, &start);
    some = hi > lo;
  }
  grid_wait();  // the pieces
  int n = 0, begin = 0;
  if (some) {
    const int2 r = runs[((long long)lane * rs.B + rg) * (Hkv * groups) + kvh * groups + hg];
    begin = r.x;
    n = r.y;
  }
  int upto = n;
  for (int s = 1; s < 32; s <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += x;
  }
  const int pieces = __shfl_sync(0xffffffffu, upto, 31);
  if (SHARDS && pieces == 1) return;
  float M = -INFINITY, wsum = 0.f, acc[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
  for (int p0 = 0; p0 < pieces; p0 += 32) {
    const int piece = p0 + lane;
    int i = 0;  // the piece's shard
    for (int s = 0; s < rs.N; ++s) i += __shfl_sync(0xffffffffu, upto, s) <= piece ? 1 : 0;
    const int ci = i < 31 ? i : 31;
    const int ni = __shfl_sync(0xffffffffu, n, ci), bi = __shfl_sync(0xffffffffu, begin, ci);
    const int j = piece - (__shfl_sync(0xffffffffu, upto, ci) - ni);  // of the shard's
    const long long row = ni == 1 ? (long long)i * rows + ro : (2ll * (bi + j) + (j == 0 ? 1 : 0)) * rows_per_lane + R;
    const float* src = (ni == 1 ? o_parts : tmp_o) + row * D;
    const float li = piece < pieces ? (ni == 1 ? lses : tmp_lse)[row] : -INFINITY;
    float mx = li;
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    mx = fmaxf(mx, M);
    if (__any_sync(0xffffffffu, li != li)) mx = 0.f;  // NaN pieces make the row NaN
    if (mx == -INFINITY) continue;
    const float old = M == -INFINITY ? 0.f : expf(M - mx);
    const float w = li == -INFINITY ? 0.f : expf(li - mx);
    M = mx;
    wsum = wsum * old + w;  // this lane's share
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] *= old;
    const int cnt = min(32, pieces - p0);
    const unsigned long long addr = reinterpret_cast<unsigned long long>(src);
#pragma unroll 4
    for (int j = 0; j < cnt; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float* sj = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, addr, j)) + kPer * lane;
      if constexpr (kPer == 4) {
        const float4 x = *reinterpret_cast<const float4*>(sj);
        acc[0] = fmaf(wj, x.x, acc[0]);
        acc[1] = fmaf(wj, x.y, acc[1]);
        acc[2] = fmaf(wj, x.z, acc[2]);
        acc[3] = fmaf(wj, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(sj);
        acc[0] = fmaf(wj, x.x, acc[0]);
        acc[1] = fmaf(wj, x.y, acc[1]);
      }
    }
  }
  for (int s = 16; s > 0; s >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, s);
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  float* dst = o + rd * D + kPer * lane;
  if constexpr (kPer == 4) *reinterpret_cast<float4*>(dst) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
  else *reinterpret_cast<float2*>(dst) = make_float2(acc[0] * inv, acc[1] * inv);
  if (lse_out && lane == 0) lse_out[rd] = wsum == 0.f ? -INFINITY : M + logf(wsum);
}

template <int D, bool HALF>
int occupancy() {
  static std::mutex mu;
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int occ = 0;
  using C = Mx4Cfg<D>;
  if (cudaFuncSetAttribute(gqa_mx4_kernel<D, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, gqa_mx4_kernel<D, HALF>, C::kThreads, C::kSmem) != cudaSuccess)
    return 0;
  if (dev < 64) cache[dev] = occ;
  return occ;
}

}  // namespace

// Query tokens of a lane: as many as its 16 rows hold.
int gqa_mx4_tokens(const dcp_attn_desc& d, int qlen) {
  const int g = d.num_q_heads / d.num_kv_heads;
  const int room = g >= 16 ? 1 : 16 / g;
  return qlen < room ? qlen : room;
}

int gqa_mx4_runs(const dcp_attn_desc& d, const DeviceInfo& di, int rows_per_lane) {
  const int occ = rows_per_lane <= 8 ? (d.head_dim_k == 128 ? occupancy<128, true>() : occupancy<64, true>())
                                     : (d.head_dim_k == 128 ? occupancy<128, false>() : occupancy<64, false>());
  return occ > 0 ? occ * di.sm_count : 0;
}

cudaError_t launch_gqa_mx4(const dcp_attn_desc& d, const void* q, const ShardSet& sh, const RangeSpec& rs,
                           float* o_parts, float* lses, void* ws, const WsLayout& L, int n_runs, int32_t* err,
                           cudaStream_t st) {
  Mx4Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.sh = sh;
  p.rs = rs;
  p.runs = reinterpret_cast<int2*>(static_cast<char*>(ws) + L.lanes_off);
  p.tmp_o = reinterpret_cast<float*>(static_cast<char*>(ws) + L.tmp_o_off);
  p.tmp_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + L.tmp_lse_off);
  p.rows_per_lane = L.rows_per_lane;
  p.o_parts = o_parts;
  p.lses = lses;
  p.err = err;
  p.ngroups = (rs.qlen + rs.tpr - 1) / rs.tpr;
  p.Bseq = rs.B / p.ngroups;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.g = d.num_q_heads / d.num_kv_heads;
  p.groups = (p.g + 15) / 16;
  p.hpl = p.g < 16 ? p.g : 16;
  p.Bs = d.block_size;
  p.sl2 = fabsf(d.scale) * kLog2e;
  p.negate = d.scale < 0.f;
  const bool half = L.rows_per_lane <= 8;
  if (d.head_dim_k == 128) {
    const auto kernel = half ? gqa_mx4_kernel<128, true> : gqa_mx4_kernel<128, false>;
    kernel<<<n_runs, Mx4Cfg<128>::kThreads, Mx4Cfg<128>::kSmem, st>>>(p);
  } else {
    const auto kernel = half ? gqa_mx4_kernel<64, true> : gqa_mx4_kernel<64, false>;
    kernel<<<n_runs, Mx4Cfg<64>::kThreads, Mx4Cfg<64>::kSmem, st>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_merge_mx4(const dcp_attn_desc& d, const RangeSpec& rs, const void* ws, const WsLayout& L,
                             float* o_parts, float* lses, float* o, float* lse_out, cudaStream_t st) {
  const int G = (rs.qlen + rs.tpr - 1) / rs.tpr;
  const long long rows = (long long)(rs.B / G) * rs.qlen * d.num_q_heads * (o ? 1 : rs.N);
  if (rows <= 0) return cudaSuccess;
  const long long grid = (rows + 3) / 4;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const char* w = static_cast<const char*>(ws);
  const int2* runs = reinterpret_cast<const int2*>(w + L.lanes_off);
  const float* tmp_o = reinterpret_cast<const float*>(w + L.tmp_o_off);
  const float* tmp_lse = reinterpret_cast<const float*>(w + L.tmp_lse_off);
  const auto kernel = d.head_dim_k == 128 ? (o ? mx4_merge_kernel<128, false> : mx4_merge_kernel<128, true>)
                                          : (o ? mx4_merge_kernel<64, false> : mx4_merge_kernel<64, true>);
  return launch_behind(kernel, (unsigned)grid, 128, 0, st, runs, tmp_o, tmp_lse, L.rows_per_lane, rs, d.num_q_heads,
                       d.num_kv_heads, (const float*)o_parts, (const float*)lses, o ? o : o_parts, o ? lse_out : lses);
}

}  // namespace dcp
