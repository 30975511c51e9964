// Accumulated attention weight per cached token.
//
// For sequence b, KV head h and cache index t, over the step's query tokens j
// (which see tokens below seq_lens[b] - (q_len - 1 - j)) and h's query heads:
//   w = sum_{j, head} exp(scale <q[b, j, head], k_t> - lse[b, j, head])
//   mass_out[b, h, t] = (t < seq_lens[b] - q_len ? mass_in[b, h, t] : 0) + w
// The softmax's denominators are known (lse), so one pass over the keys
// suffices; the scores are a product of the cached keys with the step's query
// rows and never leave the registers. Every cache index belongs to one warp:
// no atomics, and the same result on every run.
//
// Up to 16 query rows per KV head: this file. More (MLA always): the tcgen05
// kernel.
//
// On m16n8k16 MMAs the tokens are the M side (A = keys, from global memory
// straight into registers: a lane's 8 dims of every 32 are one load, and any
// order of the dims does as long as the queries' is the same) and the query
// rows the N side (B, from shared memory). 8-bit and 4-bit codes are widened to
// fp16 in registers, the queries scaled by a power of two into its range; a
// 4-bit block's scale multiplies the block's part of the dot product in fp32.
//
// Bound: HBM for bf16 (32 sequences x 32K tokens x 4 heads of 128, 16 rows,
// 1.1 GB: 179 us, 6.2 TB/s, 91 % of a plain copy; 199 us without the prefetch
// of the next tile into L2, whose loads otherwise wait for DRAM one tile at a
// time).
#include <climits>
#include <cmath>
#include <mutex>

#include "dcp_mass.cuh"
#include "dcp_mx4.cuh"

namespace dcp {
namespace {

constexpr int kMassWarps = 8;
constexpr int kMassThreads = kMassWarps * 32;

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

constexpr int kGroups = 2;          // of 8 query rows
constexpr int kRows = 8 * kGroups;

// One 32-dim chunk of a lane's dims of one token: its raw bytes.
template <int KV>
struct RawChunk {
  using T = uint4;
};
template <>
struct RawChunk<1> {
  using T = uint2;
};
template <>
struct RawChunk<2> {
  using T = uint32_t;
};

// KV: 0 bf16, 1 E4M3, 2 microscaled 4-bit.
template <int KV, int D>
__global__ void __launch_bounds__(kMassThreads) mass_kernel(const __grid_constant__ MassParams p) {
  constexpr int kChunks = D / 32;           // 32 dims: two k-steps
  constexpr int kRowBytes = D * 2 + 64;     // rows 64 bytes apart modulo 128: no bank conflict
  __shared__ __align__(128) unsigned char smem[kRows * kRowBytes];
  __shared__ float row_scale[kRows];  // score factor of a query row
  __shared__ float row_lse[kRows];    // its lse in log2 units
  __shared__ int row_lim[kRows];      // tokens it sees end here
  __shared__ RunPlace place;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, t4 = lane & 3;
  const RunPlace run = find_run<kMassThreads>(p, &place);
  const int rows = p.qlen * p.g;
  for_parts(p, run, kRows, [&](int u, int start, int n, int kvh, int t0, int t1, int) {
    const int shard = u / p.B, b = u - shard * p.B;
    const int len = p.seq_lens[b], old = len - p.qlen;
    const int32_t* table = p.sh.table[shard] + (size_t)b * p.sh.max_blocks[shard];
    const unsigned char* kpool = static_cast<const unsigned char*>(p.sh.k[shard]);
    const size_t mrow = ((size_t)b * p.Hkv + kvh) * (size_t)p.cap;
    // the query rows: row r is query token r / g, head kvh g + r % g
    __syncthreads();
#pragma unroll
    for (int r = warp; r < kRows; r += kMassWarps) {
      const int j = r / p.g;
      const bool valid = r < rows;
      const size_t qr = ((size_t)b * p.qlen + (valid ? j : 0)) * p.Hq + kvh * p.g + (valid ? r - j * p.g : 0);
      uint32_t w[D / 64];
#pragma unroll
      for (int i = 0; i < D / 64; ++i) w[i] = valid ? reinterpret_cast<const uint32_t*>(p.q + qr * D)[lane + 32 * i] : 0u;
      // a row that saw nothing weighs nothing, whatever it holds
      const float l = valid ? p.lse[qr] : -INFINITY;
      const bool some = l != -INFINITY;
      if (!some) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) w[i] = 0u;
      }
      int f = 127;
      if constexpr (KV != 0) {  // fp16 operands: the row's largest value into [1, 2)
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
        top = max(top & 0xFFFFu, top >> 16);
        for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        f = min(max((int)(top >> 7), 1), 253);
      }
      const float down = __uint_as_float((uint32_t)(254 - f) << 23);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        if constexpr (KV != 0) {
          const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
          const __half2 h = __floats2half2_rn(v.x * down, v.y * down);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint32_t*>(smem + r * kRowBytes + (lane + 32 * i) * 4) = w[i];
      }
      if (lane == 0) {
        row_scale[r] = some ? p.sl2 * __uint_as_float((uint32_t)f << 23) : 0.f;
        row_lse[r] = some ? l * kLog2e : INFINITY;
        row_lim[r] = valid ? len - (p.qlen - 1 - j) : INT_MIN;
      }
    }
    __syncthreads();

    // the block of a tile's 16 tokens of this warp, looked up a tile ahead
    auto entry = [&](int tile) -> int {
      const int base = tile * kMassTile + warp * 16, lb = base / p.Bs;
      return tile < t1 && base < n && lb < p.sh.max_blocks[shard] ? table[lb] : -1;
    };
    const int least = len - (p.qlen - 1);  // every row sees the tokens before it
    int phys_next = entry(t0);
    for (int tile = t0; tile < t1; ++tile) {
      const int base = tile * kMassTile + warp * 16;  // local index of the warp's first token
      const int phys = phys_next;
      phys_next = entry(tile + 1);
      if (base >= n) continue;
      const int lb = base / p.Bs, slot = base - lb * p.Bs;
      if (phys < 0 || phys >= p.sh.nblk[shard]) {
        if (lane == 0)
          raise_flag(p.err, lb < p.sh.max_blocks[shard] ? DCP_DEVERR_BLOCK_RANGE : DCP_DEVERR_TABLE_RANGE);
        continue;
      }
      // the next tile's keys on their way into L2: a line per lane and turn
      if (phys_next >= 0 && phys_next < p.sh.nblk[shard]) {
        const int at = base + kMassTile, slot_next = at - at / p.Bs * p.Bs;
        constexpr int kSpan = KV == 2 ? mx4_tile_codes(D) + D / 2 : 16 * D * (KV == 0 ? 2 : 1);
        const unsigned char* first = kpool + (((size_t)phys_next * p.Hkv + kvh) * p.Bs + slot_next) / 16 * (size_t)kSpan;
#pragma unroll
        for (int c = lane * 128; c < kSpan; c += 32 * 128) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(first + c));
      }
      // lanes t4 = 0 and 1 of a row write its two tokens' masses
      const int t_a = start + base + gr, t_b = t_a + 8, t_w = t4 ? t_b : t_a;
      const bool writes = t4 < 2 && t_w < start + n;
      float before_it = 0.f;
      if (writes && p.mass_in && t_w < old) before_it = p.mass_in[mrow + t_w];
      const size_t blk = (size_t)phys * p.Hkv + kvh;
      const unsigned char* tl = nullptr;   // 4-bit tile
      const unsigned char* src[2];         // the lane's bytes of its two tokens' first chunk
      constexpr int kStep = KV == 0 ? 64 : KV == 1 ? 32 : 4;  // bytes from chunk to chunk
      if constexpr (KV == 2) {
        tl = kpool + (blk * (p.Bs / kMxTile) + slot / kMxTile) * (size_t)mx4_tile_bytes(D);
        src[0] = tl + gr * (D / 2) + t4 * (D / 8);
        src[1] = src[0] + 8 * (D / 2);
      } else {
        constexpr int kElem = KV == 0 ? 2 : 1;
        src[0] = kpool + (blk * p.Bs + slot + gr) * (size_t)(D * kElem) + t4 * (8 * kElem);
        src[1] = src[0] + 8 * (size_t)(D * kElem);
      }
      float s[kGroups][4];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll 4
      for (int c = 0; c < kChunks; ++c) {
        using Raw = typename RawChunk<KV>::T;
        Raw raw[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) raw[e] = *reinterpret_cast<const Raw*>(src[e] + c * kStep);
        uint32_t a[2][4];
        float f[2] = {1.f, 1.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (KV == 0) {
            a[0][e] = raw[e].x;
            a[0][2 + e] = raw[e].y;
            a[1][e] = raw[e].z;
            a[1][2 + e] = raw[e].w;
          } else if constexpr (KV == 1) {
            e4m3x4_to_f16x4(raw[e].x, a[0][e], a[0][2 + e]);
            e4m3x4_to_f16x4(raw[e].y, a[1][e], a[1][2 + e]);
          } else {
            e2m1x8_to_f16(raw[e], a[0][e], a[0][2 + e], a[1][e], a[1][2 + e]);
            f[e] = __uint_as_float((uint32_t)tl[mx4_tile_codes(D) + (gr + 8 * e) * (D / 32) + c] << 23);
          }
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const uint4 bq = *reinterpret_cast<const uint4*>(smem + (8 * i + gr) * kRowBytes + c * 64 + t4 * 16);
          if constexpr (KV == 0) {
            mma_bf16(s[i], a[0], bq.x, bq.y);
            mma_bf16(s[i], a[1], bq.z, bq.w);
          } else if constexpr (KV == 1) {
            mma_f16(s[i], a[0], bq.x, bq.y);
            mma_f16(s[i], a[1], bq.z, bq.w);
          } else {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(acc, a[0], bq.x, bq.y);
            mma_f16(acc, a[1], bq.z, bq.w);
            s[i][0] = fmaf(f[0], acc[0], s[i][0]);
            s[i][1] = fmaf(f[0], acc[1], s[i][1]);
            s[i][2] = fmaf(f[1], acc[2], s[i][2]);
            s[i][3] = fmaf(f[1], acc[3], s[i][3]);
          }
        }
      }
      // weights, summed over the rows
      const bool masked = start + base + 16 > least;
      float wa = 0.f, wb = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * i + 2 * t4 + e;
          const float fs = row_scale[r], fl = row_lse[r];
          float ea = ex2(fmaf(s[i][e], fs, -fl)), eb = ex2(fmaf(s[i][2 + e], fs, -fl));
          if (masked) {
            const int lim = row_lim[r];
            ea = t_a < lim ? ea : 0.f;
            eb = t_b < lim ? eb : 0.f;
          }
          wa += ea;
          wb += eb;
        }
      }
      wa += __shfl_xor_sync(0xffffffffu, wa, 1);
      wa += __shfl_xor_sync(0xffffffffu, wa, 2);
      wb += __shfl_xor_sync(0xffffffffu, wb, 1);
      wb += __shfl_xor_sync(0xffffffffu, wb, 2);
      if (writes) p.mass_out[mrow + t_w] = before_it + (t4 ? wb : wa);
    }
    return true;
  });
}

template <int KV, int D>
cudaError_t launch_mass_d(const MassParams& p, int sms, cudaStream_t st) {
  static std::mutex mu;
  static int cache[64] = {};  // resident CTAs per SM
  int dev = 0, occ = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == 0) {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, mass_kernel<KV, D>, kMassThreads, 0);
      if (e != cudaSuccess || occ < 1) return cudaErrorUnknown;
      cache[dev] = occ;
    }
    occ = cache[dev];
  }
  mass_kernel<KV, D><<<sms * occ, kMassThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mass(const dcp_attn_desc& d, const ShardSet& sh, int N, const void* q, const int32_t* seq_lens,
                        const int32_t* starts, int B, int qlen, const float* lse, const float* mass_in,
                        float* mass_out, long long cap, int32_t* err, cudaStream_t st) {
  DeviceInfo di;
  if (device_info(&di) != 0) return cudaErrorUnknown;
  MassParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.sh = sh;
  p.seq_lens = seq_lens;
  p.starts = starts;
  p.lse = lse;
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.err = err;
  p.cap = cap;
  p.B = B;
  p.N = N;
  p.qlen = qlen;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.g = d.num_q_heads / d.num_kv_heads;
  p.Bs = d.block_size;
  p.sl2 = d.scale * (d.kv_dtype == DCP_KV_FP8_E4M3 ? d.k_scale : 1.f) * kLog2e;
  const int sms = di.sm_count;
  if (mass_tc_eligible(d, qlen)) return launch_mass_tc(d, p, sms, st);  // (MLA has 128 rows)
  if (d.head_dim_k == 128)
    return d.kv_dtype == DCP_KV_BF16       ? launch_mass_d<0, 128>(p, sms, st)
           : d.kv_dtype == DCP_KV_FP8_E4M3 ? launch_mass_d<1, 128>(p, sms, st)
                                           : launch_mass_d<2, 128>(p, sms, st);
  return d.kv_dtype == DCP_KV_BF16       ? launch_mass_d<0, 64>(p, sms, st)
         : d.kv_dtype == DCP_KV_FP8_E4M3 ? launch_mass_d<1, 64>(p, sms, st)
                                         : launch_mass_d<2, 64>(p, sms, st);
}

}  // namespace dcp
