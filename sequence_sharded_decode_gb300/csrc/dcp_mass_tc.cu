// Accumulated attention weight per cached token, more than 16 query rows per KV
// head (MLA's 128 heads, or a window of query tokens).
//
// S[128 tokens x rows] = K_tile . Q^T on tcgen05 with the tokens as the M side,
// so that a thread of the epilogue owns a token: it reads its scores from
// tensor memory column by column, turns them into weights exp2(s - lse) and
// adds them up without meeting another thread.
//
//   keys        64 columns of a tile (16 KB of bf16) a stage. bf16: one warp, by
//               TMA through the block table, pages that are missing read as
//               zeros. 8-bit and 4-bit: four or eight warps load codes, a
//               quarter of 64 columns of a row a lane, and store them widened
//               (both types are exact in bf16, a 4-bit value times its scale
//               too), the next tile on its way into L2 meanwhile
//   MMA warp    per tile and group of up to 128 query rows: D / 16 MMAs onto
//               one of two accumulators of 128 columns; a latent's 36 onto two
//               of four, which the epilogue adds up: the MMA's additions
//               truncate, always the same way (35 tokens x 4 x 128 rows: error
//               of the weights 1.3e-6 with one accumulator, 6e-7 with two)
//   4 warps     the epilogue; the first thread also copies the lane's query
//               rows by TMA (all four load them where the heads of a token do
//               not divide 128 or the rows 16), which stay for the lane
//
// Up to 128 kMaxQ query rows are resident and K is read once for them; more
// rows take further passes over the lane, which add to mass_out. What is
// resident sets the CTA's shared memory: up to 128 rows of a GQA head leave
// room for two CTAs an SM, whose waits and parts' starts overlap (16 x 32K x 8
// heads x 128 rows: 336 us with one CTA an SM, 209 us with two).
//
// Bounds: bf16 MLA reads 147 KB per tile, 3.3 us of an SM's share of HBM, against
// 1.3 us of MMAs (36 of 128 x 128 x 16) and 0.5 us of exponentials (128 x 128 at
// 16 a cycle): 8 x 200K tokens, 1.86 GB, 297 us (6.3 TB/s, 92 % of a plain copy).
// What stands between that and HBM is the turnover of the stages, a chain of
// short waits: with a call per wait and an election per MMA 370 us. With D =
// 128 the exponentials take 4 times the MMAs' cycles: a ragged window of 32
// tokens x 4 heads, 16 sequences of up to 8K tokens x 8 heads, 138 MB, takes 36
// us, 20 of them its bytes, 14 its exponentials; the rest is the lanes' starts.
// Widened caches are bound by the chain of load, conversion, store and turnover:
// 8 x 70K 8-bit latents 165 us with two groups of four warps (with three groups
// 154, but their registers spill and cost short sequences 6 to 15 %), 353 on
// mma.sync; the ragged window over 8 bits 59 us, over 4 bits 58.
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "dcp_mass.cuh"
#include "dcp_mx4.cuh"
#include "dcp_tc_ptx.cuh"

namespace dcp {
namespace {

constexpr int kTcRows = 128;               // tokens of a tile, and query rows of a group
constexpr int kChunkBytes = kTcRows * 128;  // 64 columns of 128 rows
constexpr int kMmaWarp = 4, kFirstCopyWarp = 5;

// KV: 0 bf16, 1 E4M3, 2 microscaled 4-bit.
template <int KV, int D>
struct MassTc {
  static constexpr int kGroups = D == 576 ? 2 : 1;              // of widening warps, which take turns at the stages
  static constexpr int kCopyWarps = KV == 0 ? 1 : 4 * kGroups;
  static constexpr int kThreads = (kFirstCopyWarp + kCopyWarps) * 32;
  static constexpr int kC = D / 64;                                // 64-column chunks of a row
  static constexpr int kParts = D == 576 ? 2 : 1;                  // accumulators of a score, added up by the epilogue
  static constexpr int kPart = (kC + kParts - 1) / kParts;         // chunks of one of them
  static constexpr int kSlots = D == 576 ? 4 : 2;                  // accumulators of 128 columns
  static constexpr int kMaxQ = D == 576 ? 1 : D == 128 ? 4 : 8;    // resident groups of 128 query rows
  static constexpr int kStages = D == 576 ? 5 : 4;
  // the resident query rows; then K stages; per query row -lse in log2 units and limit; barriers
  static constexpr int kOffRow = kStages * kChunkBytes;
  static constexpr int kOffBar = kOffRow + kMaxQ * kTcRows * 8;
  static constexpr int smem(int groups) { return groups * kC * kChunkBytes + kOffBar + 8 * (2 * kStages + 2 * kSlots + 4) + 1024; }
};

struct MassTcParams {
  CUtensorMap tm[kMaxShards];
  CUtensorMap tq;  // the query rows, if they are copied
  MassParams m;
  int box;  // tokens of a copy: divides the block size and 128
  int nq;   // resident groups of 128 query rows
  int copied_rows;  // query rows of a copy (0: the threads load them)
};

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// A warp's bounded wait whose first poll needs no call.
__device__ __forceinline__ bool wait_soon(uint32_t b, uint32_t parity, volatile int* abort_flag, int32_t* err) {
  if (kSpinLimit > 0 && __all_sync(0xffffffffu, bar_try(b, parity))) return true;
  return wait_warp(b, parity, abort_flag, err);
}
// The four MMAs of 64 columns: D (+)= A . B
__device__ __forceinline__ void mma_chunk(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n elect.sync _|e, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.u64 a1, %1, 2;\n add.u64 a2, %1, 4;\n add.u64 a3, %1, 6;\n"
      " add.u64 b1, %2, 2;\n add.u64 b2, %2, 4;\n add.u64 b3, %2, 6;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(accumulate));
}

// One copy's share of a thread that widens: 16 E4M3 codes, or 16 4-bit codes of
// two scale blocks and the blocks' scale codes.
template <int KV>
struct CodeUnit {
  uint4 w;
  __device__ __forceinline__ void load(const unsigned char* row, int c, int j) {
    w = *reinterpret_cast<const uint4*>(row + 64 * c + 16 * j);
  }
  // the pieces (eight columns each) of columns 64 c ..: e of two
  __device__ __forceinline__ static int piece(int j, int e) { return 2 * j + e; }
  __device__ __forceinline__ uint4 values(int e) const {
    const uint32_t x[2] = {e ? w.z : w.x, e ? w.w : w.y};
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h;
      asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(h) : "r"(x[i >> 1] >> (16 * (i & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      const __nv_bfloat162 z = __floats2bfloat162_rn(f.x, f.y);
      v[i] = *reinterpret_cast<const uint32_t*>(&z);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct CodeUnit<2> {
  uint2 w;
  uint32_t scales;
  template <int D>
  __device__ __forceinline__ void load_tile(const unsigned char* tile, int r, int c, int j) {
    w = *reinterpret_cast<const uint2*>(tile + r * (D / 2) + j * (D / 8) + 8 * c);
    scales = *reinterpret_cast<const unsigned short*>(tile + mx4_tile_codes(D) + r * (D / 32) + 2 * c);
  }
  __device__ __forceinline__ static int piece(int j, int e) { return j + 4 * e; }
  __device__ __forceinline__ uint4 values(int e) const {
    return mx4_widen(e ? w.y : w.x, __uint_as_float((e ? scales >> 8 : scales & 255u) << 23));
  }
};

template <int KV, int D>
__global__ void __launch_bounds__(MassTc<KV, D>::kThreads, D == 576 ? 1 : 2)
    mass_tc_kernel(const __grid_constant__ MassTcParams pp) {
  using C = MassTc<KV, D>;
  const MassParams& p = pp.m;
  extern __shared__ unsigned char smem_raw[];
  __shared__ RunPlace place;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_word;
  __shared__ volatile uint32_t left_out;  // the last part, from 1, with a row that weighs nothing
  const uint32_t raw = saddr(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t qbase = saddr(smem);
  smem += pp.nq * C::kC * kChunkBytes;
  const uint32_t sbase = saddr(smem);
  float* row_lse = reinterpret_cast<float*>(smem + C::kOffRow);
  int* row_lim = reinterpret_cast<int*>(smem + C::kOffRow + C::kMaxQ * kTcRows * 4);
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
  constexpr int BFULL = 0, BEMPTY = C::kStages, BSF = 2 * C::kStages, BSE = BSF + C::kSlots, BQF = BSE + C::kSlots, BQD = BQF + 1, BQT = BQD + 1, BDRAIN = BQT + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &abort_word;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      bar_init(bar(BFULL + s), KV == 0 ? 1 : 4 * 32);
      bar_init(bar(BEMPTY + s), 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      bar_init(bar(BSF + s), 1);
      bar_init(bar(BSE + s), kTcRows);
    }
    bar_init(bar(BQF), kTcRows);  // the part's query rows are laid out
    bar_init(bar(BQD), kTcRows);  // the part is done with: its rows may go
    bar_init(bar(BQT), 1);        // the copies of them
    bar_init(bar(BDRAIN), 1);
    abort_word = 0;
    left_out = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(saddr(&tmem_slot)), "r"(C::kSlots * 128));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  tc_fence_before();
  const RunPlace run = find_run<C::kThreads>(p, &place);  // (it synchronises the block)
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int rows = p.qlen * p.g;
  const int pass = pp.nq * kTcRows;

  if (KV != 0 && warp >= kFirstCopyWarp) {
    // ------------------------------------------------------------- widen
    // A group's warp has 32 rows of every kGroups-th stage; lane = 8 j + r:
    // quarter j of the 64 columns of rows r, r + 8, r + 16, r + 24.
    constexpr int kUnits = 4;
    constexpr int kRowBytes = KV == 1 ? D : D / 2;
    const int group = (warp - kFirstCopyWarp) / 4;
    const int j4 = lane >> 3, row0 = (warp - kFirstCopyWarp) % 4 * 32 + (lane & 7);
    uint32_t filled = 0;  // stages of all groups before the tile
    for_parts(p, run, pass, [&](int u, int start, int n, int kvh, int t0, int t1, int r0) {
      const int shard = u / p.B, b = u - shard * p.B;
      const int32_t* table = p.sh.table[shard] + (size_t)b * p.sh.max_blocks[shard];
      const unsigned char* kpool = static_cast<const unsigned char*>(p.sh.k[shard]);
      auto entry = [&](int tile, int i) -> int {
        const int at = tile * kTcRows + row0 + 8 * i, lb = at / p.Bs;
        return tile < t1 && at < n && lb < p.sh.max_blocks[shard] ? table[lb] : -1;
      };
      // the row's bytes (4-bit: those of its tile of 16 tokens), or none
      auto row_of = [&](int tile, int i, int phys) -> const unsigned char* {
        if (phys < 0 || phys >= p.sh.nblk[shard]) return nullptr;
        const int at = tile * kTcRows + row0 + 8 * i, slot = at - at / p.Bs * p.Bs;
        const size_t blk = (size_t)phys * p.Hkv + kvh;
        if constexpr (KV == 2) return kpool + (blk * (p.Bs / kMxTile) + slot / kMxTile) * (size_t)mx4_tile_bytes(D);
        else return kpool + (blk * p.Bs + slot) * (size_t)kRowBytes;
      };
      int phys[kUnits], ahead[kUnits];  // of this tile and the next
#pragma unroll
      for (int i = 0; i < kUnits; ++i) phys[i] = entry(t0, i), ahead[i] = entry(t0 + 1, i);
      for (int tile = t0; tile < t1; ++tile) {
        const unsigned char* src[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
          src[i] = row_of(tile, i, phys[i]);
          const int at = tile * kTcRows + row0 + 8 * i;
          if (!src[i] && at < n && j4 == 0 && group == 0)
            raise_flag(p.err, at / p.Bs < p.sh.max_blocks[shard] ? DCP_DEVERR_BLOCK_RANGE : DCP_DEVERR_TABLE_RANGE);
          // the next tile's row on its way into L2
          const unsigned char* after = row_of(tile + 1, i, ahead[i]);
          if (after) {
            if constexpr (KV == 2) {  // the tile's codes and scales, by the eight lanes
              const int o = (lane & 7) * 128 + j4 * 1024;
              if (o < mx4_tile_bytes(D)) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(after + o));
            } else {
              for (int o = (group * 4 + j4) * 128; o < kRowBytes; o += C::kGroups * 512) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(after + o));
            }
          }
          phys[i] = ahead[i];
          ahead[i] = entry(tile + 2, i);
        }
        for (uint32_t c = (group + filled) % C::kGroups; c < C::kC; c += C::kGroups) {
          CodeUnit<KV> code[kUnits];
#pragma unroll
          for (int i = 0; i < kUnits; ++i)
            if (src[i]) {
              if constexpr (KV == 2) code[i].template load_tile<D>(src[i], (row0 + 8 * i) & 15, c, j4);
              else code[i].load(src[i], c, j4);
            }
          const uint32_t f = filled + c, s = f % C::kStages, use = f / C::kStages;
          if (use > 0 && !wait_soon(bar(BEMPTY + s), (use - 1) & 1u, abort_flag, p.err)) return false;
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int r = row0 + 8 * i;
            if (src[i]) {  // (a row that is not there scores what it likes: nobody takes it)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint4 v = code[i].values(e);
                st_shared_v4(sbase + s * kChunkBytes + r * 128 + ((CodeUnit<KV>::piece(j4, e) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          bar_arrive(bar(BFULL + s));
        }
        filled += C::kC;
      }
      return true;
    });
  } else if (KV == 0 && warp == kFirstCopyWarp) {
    // ------------------------------------------------------------- copy
    uint32_t fills = 0;
    const int pieces = kTcRows / pp.box;
    for_parts(p, run, pass, [&](int u, int start, int n, int kvh, int t0, int t1, int r0) {
      const int shard = u / p.B, b = u - shard * p.B;
      const int32_t* table = p.sh.table[shard] + (size_t)b * p.sh.max_blocks[shard];
      // this lane's piece of a tile: its block's table entry, looked up a tile ahead
      auto entry = [&](int tile) -> int {
        const int at = tile * kTcRows + lane * pp.box, lb = at / p.Bs;
        return tile < t1 && lane < pieces && at < n && lb < p.sh.max_blocks[shard] ? table[lb] : -1;
      };
      int next = entry(t0);
      for (int tile = t0; tile < t1; ++tile) {
        int row = -pp.box;  // out of range: the copy reads zeros
        const int at = tile * kTcRows + lane * pp.box, phys = next;
        next = entry(tile + 1);
        if (lane < pieces && at < n) {
          const int lb = at / p.Bs;
          if (lb >= p.sh.max_blocks[shard]) raise_flag(p.err, DCP_DEVERR_TABLE_RANGE);
          else if (phys < 0 || phys >= p.sh.nblk[shard]) raise_flag(p.err, DCP_DEVERR_BLOCK_RANGE);
          else row = (phys * p.Hkv + kvh) * p.Bs + at - lb * p.Bs;
        }
        bool ok = true;
        for (int c = 0; c < C::kC; ++c) {
          const uint32_t s = fills % C::kStages, use = fills / C::kStages;
          if (use > 0) ok = wait_soon(bar(BEMPTY + s), (use - 1) & 1u, abort_flag, p.err);
          if (!ok) break;
          if (lane == 0) bar_arrive_tx(bar(BFULL + s), kChunkBytes);
          __syncwarp();
          if (lane < pieces)
            tma_load(sbase + s * kChunkBytes + lane * pp.box * 128, &pp.tm[shard], 64 * c, row, bar(BFULL + s));
          ++fills;
        }
        if (!ok) return false;
      }
      return true;
    });
    if (lane == 0) {  // copies in flight must land before the CTA may exit, whatever the other roles do
      const uint32_t f0 = fills > (uint32_t)C::kStages ? fills - C::kStages : 0;
      for (uint32_t f = f0; f < fills; ++f) drain_bar(bar(BFULL + f % C::kStages), (f / C::kStages) & 1u);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- MMA issue
    uint32_t stage = 0, phase = 0, groups = 0, parts = 0;  // of the tile's first stage
    const uint64_t k0 = sdesc(sbase, 0), q0 = sdesc(qbase, 0);
    for_parts(p, run, pass, [&](int u, int start, int n, int kvh, int t0, int t1, int r0) {
      if (!wait_warp(bar(BQF), parts & 1u, abort_flag, p.err)) return false;
      if ((D == 576 || pp.copied_rows) && !wait_warp(bar(BQT), parts & 1u, abort_flag, p.err)) return false;
      ++parts;
      tc_fence_after();
      const int here = min(pass, rows - r0);
      for (int tile = t0; tile < t1; ++tile) {
        uint32_t s = 0, ph = 0;
        for (int r = 0; r < here; r += kTcRows) {
          const uint32_t id = idesc(kTcRows, min(kTcRows, (here - r + 15) & ~15), 0);
          const uint64_t qd = q0 + (uint64_t)(r / kTcRows * C::kC * (kChunkBytes / 16));
          const bool last = r + kTcRows >= here;
          uint32_t buf = 0;
          s = stage, ph = phase;
#pragma unroll
          for (int c = 0; c < C::kC; ++c) {
            if (c % C::kPart == 0) {
              buf = groups % C::kSlots;
              if (groups >= C::kSlots && !wait_soon(bar(BSE + buf), (groups / C::kSlots - 1) & 1u, abort_flag, p.err)) return false;
            }
            if (r == 0 && !wait_soon(bar(BFULL + s), ph, abort_flag, p.err)) return false;
            tc_fence_after();
            mma_chunk(tmem + buf * 128u, k0 + s * (kChunkBytes / 16), qd + c * (kChunkBytes / 16), id, c % C::kPart != 0);
            if (last) mma_commit(bar(BEMPTY + s));
            if ((c + 1) % C::kPart == 0 || c + 1 == C::kC) {
              mma_commit(bar(BSF + buf));
              ++groups;
            }
            if (++s == C::kStages) s = 0, ph ^= 1u;
          }
        }
        stage = s, phase = ph;
      }
      return true;
    });
    // MMAs in flight must end before tensor memory and the stages go
    mma_commit(bar(BDRAIN));
    drain_bar(bar(BDRAIN), 0);
  } else {
    // ------------------------------------------------------------- epilogue
    uint32_t groups = 0, parts = 0, copies = 0;
    const int tid = threadIdx.x;  // 0 .. 127: the tile's token, a lane of tensor memory
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    for_parts(p, run, pass, [&](int u, int start, int n, int kvh, int t0, int t1, int r0) {
      const int shard = u / p.B, b = u - shard * p.B;
      const int len = p.seq_lens[b], old = len - p.qlen;
      const int here = min(pass, rows - r0), padded = (here + 15) & ~15;
      // the part's query rows: row r is query token r / g, head kvh g + r % g
      if (parts > 0 && !wait_warp(bar(BQD), (parts - 1) & 1u, abort_flag, p.err)) return false;
      if (D == 576 || pp.copied_rows) {
        if (tid == 0) {
          const int n_groups = (here + kTcRows - 1) / kTcRows;
          bar_arrive_tx(bar(BQT), n_groups * C::kC * pp.copied_rows * 128);
          for (int k = 0; k < n_groups * C::kC; ++k)
            tma_load3(qbase + k * kChunkBytes, &pp.tq, 64 * (k % C::kC), kvh * p.g, b * p.qlen + (r0 + k / C::kC * kTcRows) / p.g,
                      bar(BQT));
          ++copies;
        }
      } else {  // eight loads in flight per thread
        constexpr int kVec = D / 8, kAhead = 8;
        for (int i0 = tid; i0 < padded * kVec; i0 += kAhead * kTcRows) {
          uint4 v[kAhead];
#pragma unroll
          for (int m = 0; m < kAhead; ++m) {
            const int i = i0 + m * kTcRows, r = i / kVec, row = r0 + r, j = row / p.g;
            v[m] = make_uint4(0, 0, 0, 0);
            if (r < here)
              v[m] = reinterpret_cast<const uint4*>(p.q)[(((size_t)b * p.qlen + j) * p.Hq + kvh * p.g + (row - j * p.g)) * kVec +
                                                         (i - r * kVec)];
          }
#pragma unroll
          for (int m = 0; m < kAhead; ++m) {
            const int i = i0 + m * kTcRows, r = i / kVec, c = i - r * kVec;
            if (r < padded)
              st_shared_v4(qbase + ((r >> 7) * C::kC + (c >> 3)) * kChunkBytes + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4),
                           v[m].x, v[m].y, v[m].z, v[m].w);
          }
        }
      }
      for (int r = tid; r < padded; r += kTcRows) {
        const int row = r0 + r, j = row / p.g;
        float l = -INFINITY;
        if (r < here) l = p.lse[((size_t)b * p.qlen + j) * p.Hq + kvh * p.g + (row - j * p.g)];
        // a row that saw nothing weighs nothing, whatever it holds: no token is in its sight
        const bool some = l != -INFINITY;
        row_lse[r] = some ? -l * kLog2e : -INFINITY;
        row_lim[r] = some ? len - (p.qlen - 1 - j) : INT_MIN;
        if (!some && r < here) left_out = parts + 1;
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      bar_arrive(bar(BQF));
      int least = len - (p.qlen - 1 - r0 / p.g);  // every row of the part sees the tokens before it
      const int32_t* table = p.sh.table[shard] + (size_t)b * p.sh.max_blocks[shard];
      const size_t mrow = ((size_t)b * p.Hkv + kvh) * (size_t)p.cap;
      const unsigned long long scale2 = f2pack(p.sl2, p.sl2);
      // this thread's token of a tile: its block's table entry and its mass so
      // far (none for the step's own tokens), loaded a tile ahead
      auto entry = [&](int tile) -> int {
        const int local = tile * kTcRows + tid, lb = local / p.Bs;
        return tile < t1 && local < n && lb < p.sh.max_blocks[shard] ? table[lb] : -1;
      };
      auto mass = [&](int tile) -> float {
        const int local = tile * kTcRows + tid, t = start + local;
        if (tile >= t1 || local >= n) return 0.f;
        return r0 > 0 ? p.mass_out[mrow + t] : p.mass_in && t < old ? p.mass_in[mrow + t] : 0.f;
      };
      int phys = entry(t0);
      float w0 = mass(t0);
      if (!wait_warp(bar(BQF), parts & 1u, abort_flag, p.err)) return false;  // the other threads' row constants
      if (left_out == parts + 1) least = INT_MIN;  // (here: as a part of the tiles' test it cost 4 % of a ragged window)
      for (int tile = t0; tile < t1; ++tile) {
        const int t = start + tile * kTcRows + tid;
        const bool there = phys >= 0 && phys < p.sh.nblk[shard];  // else its mass_out is left alone
        const float before = w0;
        phys = entry(tile + 1);
        w0 = mass(tile + 1);
        const bool masked = start + (tile + 1) * kTcRows > least;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < here; r += kTcRows) {
          const int cols = min(kTcRows, padded - r);
          // 32 scores into weights, added to the sums
          auto add = [&](const float* v, int c) {
            const float* ls = row_lse + r + c;
            if (!masked && c + 32 <= cols) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 l = *reinterpret_cast<const float4*>(ls + i);
                float e0, e1, e2, e3;
                f2unpack(ffma2(f2pack(v[i], v[i + 1]), scale2, f2pack(l.x, l.y)), e0, e1);
                f2unpack(ffma2(f2pack(v[i + 2], v[i + 3]), scale2, f2pack(l.z, l.w)), e2, e3);
                sum[0] += ex2_ftz(e0);
                sum[1] += ex2_ftz(e1);
                sum[2] += ex2_ftz(e2);
                sum[3] += ex2_ftz(e3);
              }
            } else {
              const int* lim = row_lim + r + c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if (c + i < cols) {
                  const float e = ex2_ftz(fmaf(v[i], p.sl2, ls[i]));
                  sum[i & 3] += t < lim[i] ? e : 0.f;
                }
              }
            }
          };
#pragma unroll
          for (uint32_t k = groups; k < groups + C::kParts; ++k)
            if (!wait_soon(bar(BSF + k % C::kSlots), (k / C::kSlots) & 1u, abort_flag, p.err)) return false;
          tc_fence_after();
          for (int c = 0; c < cols; c += 32) {
            float v[32];
#pragma unroll
            for (int k = 0; k < C::kParts; ++k) {
              float w[32];
              tmem_ld32(lane_base + (groups + k) % C::kSlots * 128u + c, reinterpret_cast<uint32_t*>(w));
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = k == 0 ? w[i] : v[i] + w[i];
            }
            if (c + 32 >= cols) {
              tc_fence_before();
#pragma unroll
              for (uint32_t k = groups; k < groups + C::kParts; ++k) bar_arrive(bar(BSE + k % C::kSlots));
            }
            add(v, c);
          }
          groups += C::kParts;
        }
        if (there) p.mass_out[mrow + t] = before + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
      }
      ++parts;
      bar_arrive(bar(BQD));
      return true;
    });
    if (copies > 0) drain_bar(bar(BQT), (copies - 1) & 1u);  // a copy in flight must land before the CTA may exit
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::kSlots * 128));
  }
}

// The keys of a pool as rows of d bf16 columns; boxes of 64 columns (128
// bytes, 128-byte swizzle) by `box` rows, out-of-range rows read 0.
bool key_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t d, uint32_t box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {d, rows};
  cuuint64_t strides[1] = {d * 2};
  cuuint32_t boxes[2] = {64, box};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The query rows [tokens, heads, d]; boxes of 64 columns by the g heads of a KV head by `tokens`.
bool query_map(CUtensorMap* t, const MassParams& m, int d, int tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)m.Hq, (cuuint64_t)m.B * m.qlen};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)m.Hq * d * 2};
  cuuint32_t boxes[3] = {64, (cuuint32_t)m.g, (cuuint32_t)tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(m.q), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KV, int D>
cudaError_t launch_d(MassTcParams& p, int sms, cudaStream_t st) {
  using C = MassTc<KV, D>;
  static_assert(C::smem(C::kMaxQ) <= 232448 - 128, "shared memory of a CTA");
  static std::mutex mu;
  static int occ[64][C::kMaxQ + 1] = {};
  const int rows = p.m.qlen * p.m.g;
  p.nq = (rows + kTcRows - 1) / kTcRows;
  if (p.nq > C::kMaxQ) p.nq = C::kMaxQ;
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    n = occ[dev][p.nq];
    if (n == 0) {
      e = cudaFuncSetAttribute(mass_tc_kernel<KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(C::kMaxQ));
      if (e != cudaSuccess) return e;
      int per_sm = 0, reserved = 0;
      e = cudaDeviceGetAttribute(&per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
      if (e != cudaSuccess) return e;
      // two CTAs by shared memory, registers (launch bounds) and tensor memory
      // (256 of 512 columns each); the occupancy query answers 1 for any
      // kernel that allocates tensor memory
      n = D != 576 && 2 * (C::smem(p.nq) + reserved + 256) <= per_sm ? 2 : 1;
      occ[dev][p.nq] = n;
    }
  }
  mass_tc_kernel<KV, D><<<sms * n, C::kThreads, C::smem(p.nq), st>>>(p);
  return cudaGetLastError();
}

uint64_t pool_rows(const dcp_attn_desc& d, const ShardSet& sh, int i) {
  return (uint64_t)sh.nblk[i] * d.num_kv_heads * d.block_size;
}

}  // namespace

bool mass_tc_eligible(const dcp_attn_desc& d, int qlen) { return qlen * (d.num_q_heads / d.num_kv_heads) > 16; }

cudaError_t launch_mass_tc(const dcp_attn_desc& d, const MassParams& m, int sms, cudaStream_t st) {
  MassTcParams p;
  memset(&p, 0, sizeof(p));
  p.m = m;
  p.box = d.block_size % 64 == 0 ? 64 : d.block_size % 32 == 0 ? 32 : 16;
  // Query rows as copies of g heads by 128 / g tokens, where that makes whole
  // groups of 16 rows (a part's rows loaded by its threads: 15 us more a part
  // with D = 576, 3 us with 128).
  const int rows = m.qlen * m.g;
  if (kTcRows % m.g == 0 && rows % 16 == 0) {
    p.copied_rows = rows < kTcRows ? rows : kTcRows;
    if (!query_map(&p.tq, m, d.head_dim_k, p.copied_rows / m.g)) return cudaErrorUnknown;
  }
  if (d.kv_dtype == DCP_KV_BF16)
    for (int i = 0; i < m.N; ++i) {
      if (pool_rows(d, m.sh, i) > INT32_MAX) return cudaErrorNotSupported;  // a copy's row coordinate has 32 bits
      if (!key_map(&p.tm[i], m.sh.k[i], pool_rows(d, m.sh, i), d.head_dim_k, p.box)) return cudaErrorUnknown;
    }
  if (d.head_dim_k == 576) return d.kv_dtype == DCP_KV_BF16 ? launch_d<0, 576>(p, sms, st) : launch_d<1, 576>(p, sms, st);
  if (d.head_dim_k == 128)
    return d.kv_dtype == DCP_KV_BF16       ? launch_d<0, 128>(p, sms, st)
           : d.kv_dtype == DCP_KV_FP8_E4M3 ? launch_d<1, 128>(p, sms, st)
                                           : launch_d<2, 128>(p, sms, st);
  return d.kv_dtype == DCP_KV_BF16       ? launch_d<0, 64>(p, sms, st)
         : d.kv_dtype == DCP_KV_FP8_E4M3 ? launch_d<1, 64>(p, sms, st)
                                         : launch_d<2, 64>(p, sms, st);
}

}  // namespace dcp
