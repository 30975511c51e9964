// Rows of the paged cache as bf16: quantising append into the microscaled
// 4-bit cache, and read-back of any cache's rows.
//
// Both are copies with a little arithmetic per value (a maximum over 32
// values and a rounding, or a widening): bound by the bf16 side's bytes, four
// times the codes', as long as a lane has eight values of a row (with four, the
// instructions of the append were the bound: 81 us where it takes 62 now). With
// few tokens per sequence (a decode step) one warp takes a row of one KV head.
// With many (a prompt) neighbouring tokens share a 4-bit tile, and a warp takes
// a tile of one KV head: the tokens of the call are cut into windows of 16, each of which handles the runs (consecutive
// tokens of one tile) that begin in it, so the order of the tokens does not
// matter for the result, and usual orders give whole tiles. The value codes of
// a whole tile are transposed in shared memory and stored as they lie in the
// pool instead of by atomics. 8 x 8192 tokens of 8 heads of 128 dims, 339 MB
// either way: append 62 us (5.5 TB/s), read 58 us (5.8 TB/s); four loads of 16
// bytes of keys and of values in flight a lane (two: 6 us more, eight: 10).
#include "dcp_mx4.cuh"

namespace dcp {
namespace {

constexpr int kRowThreads = 128;

struct RowParams {
  ShardSet sh;
  const int32_t* starts;
  const int32_t* seq_ids;
  const int32_t* positions;
  const void* k_new;  // append: bf16 rows in
  const void* v_new;
  void* k_out;        // read: bf16 rows out
  void* v_out;
  int32_t* err;
  int N, B, T, Hkv, Bs, D, Dv;
  float k_scale, v_scale;
};

// Where a token's row is.
struct Place {
  int owner;      // shard; -1: no place (the device error flag says why)
  int slot;       // within the block
  long long phys;
};
__device__ __forceinline__ Place row_place(const RowParams& p, long long tok, bool report) {
  Place w = {-1, 0, 0};
  const int b = p.seq_ids ? p.seq_ids[tok] : (int)tok;
  const int t = p.positions[tok];
  int o = -1;
  if (b >= 0 && b < p.B && t >= 0) {
    const int32_t* st = p.starts + (size_t)b * p.N;
    for (int i = 0; i < p.N; ++i)
      if (st[i] <= t) o = i;
  }
  if (o < 0) {
    if (report) raise_flag(p.err, DCP_DEVERR_POSITION);
    return w;
  }
  const int local = t - p.starts[(size_t)b * p.N + o];
  const int lb = local / p.Bs;
  if (lb >= p.sh.max_blocks[o]) {
    if (report) raise_flag(p.err, DCP_DEVERR_TABLE_RANGE);
    return w;
  }
  const int ph = p.sh.table[o][(size_t)b * p.sh.max_blocks[o] + lb];
  if (ph < 0 || ph >= p.sh.nblk[o]) {
    if (report) raise_flag(p.err, DCP_DEVERR_BLOCK_RANGE);
    return w;
  }
  w.owner = o;
  w.phys = ph;
  w.slot = local - lb * p.Bs;
  return w;
}

// A warp's window of the call's tokens: lane l looks at token first - 1 + l,
// tokens first .. first + 15 are its own. Runs that begin in it are lanes of
// `starts`; the run of lane l is `length(l)` tokens of one tile, in order.
struct Window {
  long long first;
  Place mine;
  unsigned starts, follows;  // follows: the lane's token continues the run of the lane before
  __device__ __forceinline__ int length(int l) const { return l == 31 ? 1 : __ffs(~(follows >> (l + 1))); }
};
__device__ __forceinline__ Window window_of(const RowParams& p, long long w) {
  const int lane = threadIdx.x & 31;
  Window x;
  x.first = w * kMxTile;
  const long long tok = x.first - 1 + lane;
  x.mine = {-1, 0, 0};
  if (tok >= 0 && tok < p.T) x.mine = row_place(p, tok, blockIdx.y == 0 && lane >= 1 && lane <= 16);
  const int owner = __shfl_up_sync(0xffffffffu, x.mine.owner, 1), slot = __shfl_up_sync(0xffffffffu, x.mine.slot, 1);
  const long long phys = __shfl_up_sync(0xffffffffu, x.mine.phys, 1);
  const bool next = lane > 0 && x.mine.owner >= 0 && owner == x.mine.owner && phys == x.mine.phys &&
                    x.mine.slot == slot + 1 && x.mine.slot % kMxTile != 0;
  x.follows = __ballot_sync(0xffffffffu, next);
  x.starts = __ballot_sync(0xffffffffu, x.mine.owner >= 0 && !next) & 0x1FFFEu;
  return x;
}

// Eight consecutive values of a row of D: D / 8 lanes take a row.
__device__ __forceinline__ uint4 load_part(const void* rows, size_t row, int per_row, int x) {
  return reinterpret_cast<const uint4*>(rows)[row * per_row + x];
}

// The codes of a lane's eight values, a nibble each, and the scale code of
// their block (four neighbouring lanes'). The magnitudes of bf16 values order
// like their 15 low bits, so the block's maximum is taken on packed 16-bit
// integers. For the whole warp at once.
__device__ __forceinline__ uint32_t quantise(uint4 part, int* scale, bool* odd) {
  const uint32_t w[4] = {part.x, part.y, part.z, part.w};
  float x[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
    top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
  }
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  top = max(top & 0xFFFFu, top >> 16);
  uint32_t q = 0;
  if (__any_sync(0xffffffffu, top >= 0x7F80u)) {  // infinities or NaN: the finite values set the scale
    *odd = *odd || top >= 0x7F80u;
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = (__float_as_uint(x[i]) >> 16) & 0x7FFFu;
      top = a < 0x7F80u && a > top ? a : top;
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int c = mx4_scale_code(top << 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) q |= mx4_code(x[i], c) << (4 * i);
    *scale = c;
    return q;
  }
  *scale = mx4_scale_code(top << 16);
  return mx4_code_eight(x, *scale);
}

// Lane x of a key row: its eight dims are one word of the tile.
template <int D>
__device__ __forceinline__ void store_key(unsigned char* tile, int r, uint32_t q, int x) {
  *reinterpret_cast<uint32_t*>(tile + r * (D / 2) + (x % 4) * (D / 8) + (x / 4) * 4) = q;
}
template <int D>
__device__ __forceinline__ void store_scale(unsigned char* tile, int r, int c, int x) {
  if (x % 4 == 0) tile[mx4_tile_codes(D) + r * (D / 32) + x / 4] = (unsigned char)c;
}
// A single value row: a lane has the four dims of a word (8 apart; word w of
// the region of dims 8 m + gr) and sets its token's nibbles. eight(i): the
// codes of dims 8 i .. 8 i + 7.
template <int D, class F>
__device__ __forceinline__ void store_value(unsigned char* tile, int r, int lane, F eight) {
  constexpr int kPer = D / 32;
  const int gr = lane / kPer % 8, w = lane % kPer;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) word |= ((eight(4 * w + i) >> (4 * gr)) & 15u) << (8 * i);
  if (lane < 8 * kPer) {
    const int n4 = 4 * (r & 1);
    unsigned int* dst = reinterpret_cast<unsigned int*>(tile + (r / 8) * (4 * D) + (gr * 4 + (r % 8) / 2) * (D / 8)) + w;
    atomicAnd(dst, ~(0x0F0F0F0Fu << n4));
    atomicOr(dst, word << n4);
  }
}
// The value codes of a whole tile, from rows of D / 2 bytes (a nibble a dim) in
// shared memory. A lane takes two neighbouring tokens and 32 dims: nibbles of
// the two rows meet in bytes, and two transpositions of 4 x 4 bytes turn the
// bytes of four groups of 8 dims into the words of 8 regions.
template <int D>
__device__ __forceinline__ void store_value_tile(unsigned char* tile, const unsigned char* rows, int pitch, int lane) {
  constexpr int kX = D / 32;
  const int x = lane % kX, t4 = lane / kX % 4, half = lane / (4 * kX);
  if (half > 1) return;  // D = 64: half the lanes
  const uint4 a = *reinterpret_cast<const uint4*>(rows + (8 * half + 2 * t4) * pitch + 16 * x);
  const uint4 b = *reinterpret_cast<const uint4*>(rows + (8 * half + 2 * t4 + 1) * pitch + 16 * x);
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int odd = 0; odd < 2; ++odd) {
    uint32_t e[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
      e[m] = odd ? ((wa[m] >> 4) & 0x0F0F0F0Fu) | (wb[m] & 0xF0F0F0F0u) : (wa[m] & 0x0F0F0F0Fu) | ((wb[m] & 0x0F0F0F0Fu) << 4);
    const uint32_t p0 = __byte_perm(e[0], e[1], 0x5140), p1 = __byte_perm(e[0], e[1], 0x7362);
    const uint32_t p2 = __byte_perm(e[2], e[3], 0x5140), p3 = __byte_perm(e[2], e[3], 0x7362);
    const uint32_t out[4] = {__byte_perm(p0, p2, 0x5410), __byte_perm(p0, p2, 0x7632), __byte_perm(p1, p3, 0x5410),
                             __byte_perm(p1, p3, 0x7632)};
#pragma unroll
    for (int j = 0; j < 4; ++j)  // byte j of e: dim 2 j + odd of each group
      *reinterpret_cast<uint32_t*>(tile + half * 4 * D + ((2 * j + odd) * 4 + t4) * (D / 8) + 4 * x) = out[j];
  }
}
// One warp per (token, KV head): D / 8 lanes the key row, as many the value row.
template <int D>
__global__ void __launch_bounds__(kRowThreads) mx4_append_kernel(const __grid_constant__ RowParams p) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const long long tok = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (tok >= p.T) return;
  const int part = lane / kLanes, x = lane % kLanes;
  const uint4 mine = load_part(part == 0 ? p.k_new : p.v_new, (size_t)tok * p.Hkv + h, kLanes, x);
  const Place at = row_place(p, tok, lane == 0 && h == 0);
  if (at.owner < 0) return;
  const int r = at.slot % kMxTile;
  unsigned char* kt = mx4_tile(const_cast<void*>(p.sh.k[at.owner]), at.phys, p.Hkv, h, p.Bs, D, at.slot);
  unsigned char* vt = mx4_tile(const_cast<void*>(p.sh.v[at.owner]), at.phys, p.Hkv, h, p.Bs, D, at.slot);
  bool odd = false;
  int c;
  const uint32_t q = quantise(mine, &c, &odd);
  if (part == 0) store_key<D>(kt, r, q, x);
  if (part < 2) store_scale<D>(part == 0 ? kt : vt, r, c, x);
  store_value<D>(vt, r, lane, [&](int i) { return __shfl_sync(0xffffffffu, q, kLanes + i); });
  if (__any_sync(0xffffffffu, odd) && lane == 0) raise_flag(p.err, DCP_DEVERR_NONFINITE);
}

// One warp per (window of 16 tokens, KV head).
template <int D>
__global__ void __launch_bounds__(kRowThreads) mx4_append_tiles_kernel(const __grid_constant__ RowParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a step
  constexpr int kAhead = 4;                           // steps loaded at a time
  constexpr int kPitch = D / 2 + 32;                  // (two rows 64 bytes apart modulo 128: no bank conflict)
  __shared__ __align__(16) unsigned char stage[kRowThreads / 32][kMxTile * kPitch];  // value codes of a tile
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const long long w = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (w * kMxTile >= p.T) return;
  const int sub = lane / kLanes, x = lane % kLanes;
  unsigned char* mine = stage[threadIdx.x >> 5];
  const Window win = window_of(p, w);
  bool odd = false;
  for (unsigned left = win.starts; left; left &= left - 1) {
    const int l = __ffs(left) - 1, n = win.length(l);
    const int owner = __shfl_sync(0xffffffffu, win.mine.owner, l), slot = __shfl_sync(0xffffffffu, win.mine.slot, l);
    const long long phys = __shfl_sync(0xffffffffu, win.mine.phys, l);
    unsigned char* kt = mx4_tile(const_cast<void*>(p.sh.k[owner]), phys, p.Hkv, h, p.Bs, D, slot);
    unsigned char* vt = mx4_tile(const_cast<void*>(p.sh.v[owner]), phys, p.Hkv, h, p.Bs, D, slot);
    const int r0 = slot % kMxTile;
    const size_t row0 = (size_t)(win.first - 1 + l) * p.Hkv + h;
    __syncwarp();
    for (int i0 = 0; i0 < n; i0 += kAhead * kRows) {
      uint4 k[kAhead], v[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const size_t row = row0 + (size_t)min(i0 + a * kRows + sub, n - 1) * p.Hkv;
        k[a] = load_part(p.k_new, row, kLanes, x);
        v[a] = load_part(p.v_new, row, kLanes, x);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int i = i0 + a * kRows + sub, r = r0 + i;
        int ck, cv;
        const uint32_t qk = quantise(k[a], &ck, &odd), qv = quantise(v[a], &cv, &odd);
        if (i < n) {
          store_key<D>(kt, r, qk, x);
          store_scale<D>(kt, r, ck, x);
          store_scale<D>(vt, r, cv, x);
          *reinterpret_cast<uint32_t*>(mine + r * kPitch + 4 * x) = qv;
        }
      }
    }
    __syncwarp();
    if (n == kMxTile) store_value_tile<D>(vt, mine, kPitch, lane);
    else
      for (int r = r0; r < r0 + n; ++r)
        store_value<D>(vt, r, lane, [&](int i) { return *reinterpret_cast<const uint32_t*>(mine + r * kPitch + 4 * i); });
  }
  if (__any_sync(0xffffffffu, odd) && lane == 0) raise_flag(p.err, DCP_DEVERR_NONFINITE);
}

__device__ __forceinline__ float e4m3_value(unsigned char code) {
  uint32_t h;
  asm("{\n .reg .b16 a;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(h) : "r"((uint32_t)code));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

// The D / 32 dims of a lane of a 4-bit key row, as bf16.
template <int D>
__device__ __forceinline__ void read_key(const unsigned char* tile, int r, int lane, __nv_bfloat16* out) {
  constexpr int kPer = D / 32;
  const int d0 = kPer * lane;
  const unsigned char* s = tile + r * (D / 2) + ((d0 % 32) / 8) * (D / 8) + (d0 / 32) * 4 + (d0 % 8) / 2;
  const uint32_t c = tile[mx4_tile_codes(D) + r * kPer + d0 / 32];
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(mx4_value(s[i], c), mx4_value(s[i] >> 4, c));
    w[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  if constexpr (D == 128) reinterpret_cast<uint2*>(out)[lane] = make_uint2(w[0], w[1]);
  else reinterpret_cast<uint32_t*>(out)[lane] = w[0];
}

// A product for a further rounding: of the two fp32 values around it the odd one
// (or itself), which no coarser format has a tie at, so that rounding it to bf16
// rounds the exact product (28 bits) once.
__device__ __forceinline__ float mul_odd(float a, float b) {
  const float lo = __fmul_rd(a, b), hi = __fmul_ru(a, b);
  return __float_as_uint(lo) & 1u ? lo : hi;
}

// Four E4M3 codes times a scale as four bf16 values.
__device__ __forceinline__ uint2 e4m3_widen(uint32_t codes, float scale) {
  uint32_t h[2], v[2];
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const __nv_bfloat162 z = __floats2bfloat162_rn(mul_odd(scale, f.x), mul_odd(scale, f.y));
    v[i] = *reinterpret_cast<const uint32_t*>(&z);
  }
  return make_uint2(v[0], v[1]);
}

// bf16 (KV 0) and E4M3 (1) rows, one warp per (32 tokens, KV head; 8 latents,
// whose rows are long and whose heads are one): a lane looks up a token, then the rows' 16-byte pieces are laid end to end over the
// lanes, four in flight. 8-bit values lie transposed in their block: a lane each
// token, whose neighbours' bytes lie beside its own. D 576: latent rows. 8 x 8192
// tokens of 8 heads of 128 dims: bf16 93 us (79 of bytes; a warp per row 178),
// 8-bit 169 us (59; 388), bound by the values' single bytes; latents 32 and 27 us
// (22 and 17; 41 and 83). Products rounded twice would save 4 and 2 us of the
// 8-bit ones.
constexpr int rows_tokens(int d) { return d == 576 ? 8 : 32; }
template <int KV, int D>
__global__ void __launch_bounds__(kRowThreads) read_rows_kernel(const __grid_constant__ RowParams p) {
  constexpr int kRow = KV == 0 ? 2 * D : D, kPieces = kRow / 16, kAhead = 4, kTokens = rows_tokens(D);
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const long long tok0 = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kTokens;
  if (tok0 >= p.T) return;
  Place at = {-1, 0, 0};
  if (lane < kTokens && tok0 + lane < p.T) at = row_place(p, tok0 + lane, h == 0);
  const size_t blk = (size_t)at.phys * p.Hkv + h;
#pragma unroll
  for (int side = 0; side < (D == 576 ? 1 : 2); ++side) {
    unsigned char* out = static_cast<unsigned char*>(side ? p.v_out : p.k_out);
    const float scale = side ? p.v_scale : p.k_scale;
    const unsigned char* pool = nullptr;
    if (at.owner >= 0) pool = static_cast<const unsigned char*>(side ? p.sh.v[at.owner] : p.sh.k[at.owner]);
    if (KV == 1 && side == 1) {
      if (pool) {
        const unsigned char* src = pool + blk * p.Bs * D + at.slot;
        uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)(tok0 + lane) * p.Hkv + h) * (2 * D));
#pragma unroll 2
        for (int d = 0; d < D; d += 8) {
          uint32_t w[2] = {0u, 0u};
#pragma unroll
          for (int a = 0; a < 8; ++a) w[a / 4] |= (uint32_t)src[(d + a) * p.Bs] << (8 * (a % 4));
          const uint2 x = e4m3_widen(w[0], scale), y = e4m3_widen(w[1], scale);
          dst[d / 8] = make_uint4(x.x, x.y, y.x, y.y);
        }
      }
      continue;
    }
    const unsigned long long mine = pool ? reinterpret_cast<unsigned long long>(pool + (blk * p.Bs + at.slot) * (size_t)kRow) : 0ull;
    for (int x0 = lane; x0 < kTokens * kPieces + lane; x0 += 32 * kAhead) {
      uint4 piece[kAhead];
      bool there[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int x = x0 + 32 * a, m = x / kPieces, c = x - m * kPieces;
        const unsigned long long src = __shfl_sync(0xffffffffu, mine, m & 31);
        there[a] = src != 0ull && m < kTokens;
        if (there[a]) piece[a] = reinterpret_cast<const uint4*>(src)[c];
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int x = x0 + 32 * a, m = x / kPieces, c = x - m * kPieces;
        if (!there[a]) continue;
        uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)(tok0 + m) * p.Hkv + h) * (2 * D));
        if constexpr (KV == 0) {
          dst[c] = piece[a];
        } else {
          const uint2 x0v = e4m3_widen(piece[a].x, scale), x1 = e4m3_widen(piece[a].y, scale);
          const uint2 x2 = e4m3_widen(piece[a].z, scale), x3 = e4m3_widen(piece[a].w, scale);
          dst[2 * c] = make_uint4(x0v.x, x0v.y, x1.x, x1.y);
          dst[2 * c + 1] = make_uint4(x2.x, x2.y, x3.x, x3.y);
        }
      }
    }
  }
}

// One warp per (token, KV head). KV: 0 bf16, 1 E4M3, 2 microscaled 4-bit.
template <int KV>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const __grid_constant__ RowParams p) {
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const long long tok = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (tok >= p.T) return;
  const Place at = row_place(p, tok, lane == 0 && h == 0);
  if (at.owner < 0) return;
  const int D = p.D, slot = at.slot;
  const size_t blk = (size_t)at.phys * p.Hkv + h;
  for (int side = 0; side < (p.v_out ? 2 : 1); ++side) {
    const unsigned char* pool = static_cast<const unsigned char*>(side ? p.sh.v[at.owner] : p.sh.k[at.owner]);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(side ? p.v_out : p.k_out) + ((size_t)tok * p.Hkv + h) * D;
    if constexpr (KV == 0) {
      const uint4* src = reinterpret_cast<const uint4*>(pool + (blk * p.Bs + slot) * D * 2);
      for (int c = lane; c < D / 8; c += 32) reinterpret_cast<uint4*>(out)[c] = src[c];
    } else if constexpr (KV == 1) {
      const float scale = side ? p.v_scale : p.k_scale;
      const unsigned char* src = pool + blk * p.Bs * D;
      for (int d = lane; d < D; d += 32)
        out[d] = __float2bfloat16(mul_odd(scale, e4m3_value(side ? src[(size_t)d * p.Bs + slot] : src[(size_t)slot * D + d])));
    } else {
      const unsigned char* t = mx4_tile(const_cast<unsigned char*>(pool), at.phys, p.Hkv, h, p.Bs, D, slot);
      const int r = slot % kMxTile;
      if (side) {
        for (int d = 2 * lane; d < D; d += 64) {
          const uint32_t c = t[mx4_tile_codes(D) + r * (D / 32) + d / 32];
          const unsigned char* s = t + (r / 8) * (4 * D) + ((d % 8) * 4 + (r % 8) / 2) * (D / 8) + d / 8;
          *reinterpret_cast<__nv_bfloat162*>(out + d) = __floats2bfloat162_rn(
              mx4_value(s[0] >> (4 * (r & 1)), c), mx4_value(s[D / 2] >> (4 * (r & 1)), c));
        }
      } else if (D == 128) {
        read_key<128>(t, r, lane, out);
      } else {
        read_key<64>(t, r, lane, out);
      }
    }
  }
}

// 4-bit rows, one warp per (window of 16 tokens, KV head). A lane widens one
// scale block of two neighbouring tokens; values take the way back through the
// append's transpositions. Rows leave through shared memory, so that a store
// covers whole rows.
template <int D>
__global__ void __launch_bounds__(kRowThreads) mx4_read_tiles_kernel(const __grid_constant__ RowParams p) {
  constexpr int kX = D / 32, kRow = 2 * D, kPitch = kRow + 16, kChunks = kRow / 16;
  __shared__ __align__(16) unsigned char stage[kRowThreads / 32][kMxTile * kPitch];
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const long long w = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (w * kMxTile >= p.T) return;
  unsigned char* mine = stage[threadIdx.x >> 5];
  const Window win = window_of(p, w);
  // this lane's scale block and tokens 8 half + 2 t4, + 1 (D = 64: half the lanes have one)
  const int x = lane % kX, t4 = lane / kX % 4, half = lane / (4 * kX), tok = 8 * half + 2 * t4;
  const bool has = half < 2;
  for (unsigned left = win.starts; left; left &= left - 1) {
    const int l = __ffs(left) - 1, n = win.length(l);
    const int owner = __shfl_sync(0xffffffffu, win.mine.owner, l), slot = __shfl_sync(0xffffffffu, win.mine.slot, l);
    const long long phys = __shfl_sync(0xffffffffu, win.mine.phys, l);
    const unsigned char* kt = mx4_tile(const_cast<void*>(p.sh.k[owner]), phys, p.Hkv, h, p.Bs, D, slot);
    const unsigned char* vt = mx4_tile(const_cast<void*>(p.sh.v[owner]), phys, p.Hkv, h, p.Bs, D, slot);
    const int r0 = slot % kMxTile;
    const size_t row0 = (size_t)(win.first - 1 + l) * p.Hkv + h;
    uint32_t kw[2][4], vw[8];
    float kf[2], vf[2];
    if (has) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        vw[j] = *reinterpret_cast<const uint32_t*>(vt + half * 4 * D + (j * 4 + t4) * (D / 8) + 4 * x);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int m = 0; m < 4; ++m) kw[e][m] = *reinterpret_cast<const uint32_t*>(kt + (tok + e) * (D / 2) + m * (D / 8) + 4 * x);
        kf[e] = __uint_as_float((uint32_t)kt[mx4_tile_codes(D) + (tok + e) * kX + x] << 23);
        vf[e] = __uint_as_float((uint32_t)vt[mx4_tile_codes(D) + (tok + e) * kX + x] << 23);
      }
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncwarp();
      if (has) {
        if (side) {  // regions' words (dim 8 m + gr of two tokens) to rows' words (8 dims of a token)
          uint32_t b[2][4];
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t p0 = __byte_perm(vw[odd], vw[odd + 2], 0x5140), p1 = __byte_perm(vw[odd], vw[odd + 2], 0x7362);
            const uint32_t p2 = __byte_perm(vw[odd + 4], vw[odd + 6], 0x5140), p3 = __byte_perm(vw[odd + 4], vw[odd + 6], 0x7362);
            b[odd][0] = __byte_perm(p0, p2, 0x5410);
            b[odd][1] = __byte_perm(p0, p2, 0x7632);
            b[odd][2] = __byte_perm(p1, p3, 0x5410);
            b[odd][3] = __byte_perm(p1, p3, 0x7632);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            kw[0][m] = (b[0][m] & 0x0F0F0F0Fu) | ((b[1][m] & 0x0F0F0F0Fu) << 4);
            kw[1][m] = ((b[0][m] >> 4) & 0x0F0F0F0Fu) | (b[1][m] & 0xF0F0F0F0u);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int m = 0; m < 4; ++m)
            *reinterpret_cast<uint4*>(mine + (tok + e) * kPitch + 64 * x + 16 * m) = mx4_widen(kw[e][m], side ? vf[e] : kf[e]);
      }
      __syncwarp();
      unsigned char* out = static_cast<unsigned char*>(side ? p.v_out : p.k_out);
#pragma unroll
      for (int i = 0; i < kMxTile * kChunks / 32; ++i) {
        const int r = (i * 32 + lane) / kChunks, c = lane % kChunks;
        if (r >= r0 && r < r0 + n)
          *reinterpret_cast<uint4*>(out + (row0 + (size_t)(r - r0) * p.Hkv) * kRow + 16 * c) =
              *reinterpret_cast<const uint4*>(mine + r * kPitch + 16 * c);
      }
    }
  }
}

RowParams row_params(const dcp_attn_desc& d, const ShardSet& sh, int N, const int32_t* starts, int B,
                     const int32_t* seq_ids, const int32_t* positions, int T, int32_t* err) {
  RowParams p;
  p.sh = sh;
  p.starts = starts;
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.k_new = p.v_new = nullptr;
  p.k_out = p.v_out = nullptr;
  p.err = err;
  p.N = N;
  p.B = B;
  p.T = T;
  p.Hkv = d.num_kv_heads;
  p.Bs = d.block_size;
  p.D = d.head_dim_k;
  p.Dv = d.head_dim_v;
  p.k_scale = d.kv_dtype == DCP_KV_FP8_E4M3 ? d.k_scale : 1.f;
  p.v_scale = d.kv_dtype == DCP_KV_FP8_E4M3 ? d.v_scale : 1.f;
  return p;
}

// Warps of `work` (tokens or windows) by KV heads.
dim3 row_grid(long long work, int heads) {
  return dim3((unsigned)((work + kRowThreads / 32 - 1) / (kRowThreads / 32)), (unsigned)heads);
}
// Many tokens per sequence: neighbours share tiles. Append and read of 8 heads
// of 128 dims, a warp per row against a warp per tile: 2 tokens of 2048
// sequences 33 / 47 us, 4 of 512 22 / 29 (of 2048: 57 / 50), 8 of 512 33 / 26,
// 16 of 512 55 / 30, 8192 of 8 400 / 121.
bool by_tiles(const RowParams& p) { return p.T >= 8LL * p.B; }
long long windows(int T) { return ((long long)T + kMxTile - 1) / kMxTile; }

}  // namespace

cudaError_t launch_append_mx4(const dcp_attn_desc& d, const ShardSet& sh, int N, const int32_t* starts, int B,
                              const int32_t* seq_ids, const int32_t* positions, const void* k_new, const void* v_new,
                              int T, int32_t* err, cudaStream_t st) {
  if (T <= 0) return cudaSuccess;
  RowParams p = row_params(d, sh, N, starts, B, seq_ids, positions, T, err);
  p.k_new = k_new;
  p.v_new = v_new;
  if (by_tiles(p)) {
    const dim3 grid = row_grid(windows(T), p.Hkv);
    if (d.head_dim_k == 128) mx4_append_tiles_kernel<128><<<grid, kRowThreads, 0, st>>>(p);
    else mx4_append_tiles_kernel<64><<<grid, kRowThreads, 0, st>>>(p);
  } else {
    const dim3 grid = row_grid(T, p.Hkv);
    if (d.head_dim_k == 128) mx4_append_kernel<128><<<grid, kRowThreads, 0, st>>>(p);
    else mx4_append_kernel<64><<<grid, kRowThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_read(const dcp_attn_desc& d, const ShardSet& sh, int N, const int32_t* starts, int B,
                        const int32_t* seq_ids, const int32_t* positions, void* k_out, void* v_out, int T, int32_t* err,
                        cudaStream_t st) {
  if (T <= 0) return cudaSuccess;
  RowParams p = row_params(d, sh, N, starts, B, seq_ids, positions, T, err);
  p.k_out = k_out;
  p.v_out = v_out;
  const dim3 grid = row_grid(T, p.Hkv);
  if (d.kv_dtype == DCP_KV_MXFP4 && by_tiles(p)) {
    const dim3 tiles = row_grid(windows(T), p.Hkv);
    if (d.head_dim_k == 128) mx4_read_tiles_kernel<128><<<tiles, kRowThreads, 0, st>>>(p);
    else mx4_read_tiles_kernel<64><<<tiles, kRowThreads, 0, st>>>(p);
  } else if (by_tiles(p)) {
    const int each = rows_tokens(d.head_dim_k);
    const dim3 rows = row_grid(((long long)T + each - 1) / each, p.Hkv);
    const bool f8 = d.kv_dtype == DCP_KV_FP8_E4M3;
    auto kernel = f8 ? read_rows_kernel<1, 576> : read_rows_kernel<0, 576>;
    if (d.head_dim_k == 128) kernel = f8 ? read_rows_kernel<1, 128> : read_rows_kernel<0, 128>;
    else if (d.head_dim_k == 64) kernel = f8 ? read_rows_kernel<1, 64> : read_rows_kernel<0, 64>;
    kernel<<<rows, kRowThreads, 0, st>>>(p);
  } else if (d.kv_dtype == DCP_KV_MXFP4) {
    read_kernel<2><<<grid, kRowThreads, 0, st>>>(p);
  } else if (d.kv_dtype == DCP_KV_FP8_E4M3) {
    read_kernel<1><<<grid, kRowThreads, 0, st>>>(p);
  } else {
    read_kernel<0><<<grid, kRowThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace dcp
