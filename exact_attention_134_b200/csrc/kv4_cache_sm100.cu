// kv4_cache_sm100.cu — writing, reading back and copying pages of the 4-bit
// key/value cache (records and page table: kv4_format.cuh).
//
// Quantisation, for a token, kv head and group of 32 channels x_c (bf16):
//   lo = min_c x_c (a bf16 number itself, so exact), s = bf16((max - lo) / 15),
//   code_c = round((x_c - lo) / s), ties to even (15 at most: s is at least
//   (1 - 2^-8) (max - lo) / 15);
// the cache then stands for lo + s * code_c, off by at most s / 2 + 15 * 2^-8 s.
// A group whose spread is below 15 * 2^-125 is held as its minimum (codes of 0;
// its scale is 2^-13 of the minimum's size, below which no spread of bf16
// values leads, so that attention can bound its weights by scales alone). A
// group with a NaN or an infinity is held as NaN (s = NaN, lo = 0).
//
// HBM-bound: 5.25 d bytes a token and head each way (bf16 against 5 bits). The
// quotients took most of the instructions: a division and comparisons for the
// ties cost 24 instructions a value; the reciprocal, one Newton step (which
// makes every quotient that is exact in fp32, a tie above all, exact) and the
// rounding by adding 1.5 * 2^23 are 9, on the FMA pipe, two values each.
// Measured (B200), 4 x 2048 new tokens of 8 heads of 128 and all 64000 read
// back: one thread per 8 values 190 us, a warp per record 106, both sides in
// warps of their own 80, quotients as above 75 (the bytes take 59); 250 single
// tokens and back 10 us.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attn_internal.h"
#include "kv4_format.cuh"
#include "sm100_rows.cuh"

namespace attn_sm100 {
namespace {

constexpr int kThreads = 256;

struct AppendParams {
  Kv4Pool c;
  uint8_t* pool;
  const uint16_t* x[2];    // k, v
  long long ts[2], hs[2];  // their token and head strides (elements)
  int* status;
};

// A warp has one record: lane 4 r + t holds 8 channels, 32 g + 8 t onwards, of
// the tokens r and r + 8 in every group g. Those are its K words; a V word is
// half the lane's own and half its neighbour's of the other token of a pair
// (lane ^ 4), so one exchange turns one order into the other. A block is one
// item (16 tokens of a sequence), its warps are heads and sides.

// The record of an item and head, or null: no page of the pool.
__device__ __forceinline__ size_t record_at(const Kv4Pool& c, const Kv4Item& t, int h, int d, int* status, int where,
                                            bool& ok) {
  const int page = __ldg(c.table + (size_t)t.b * c.max_pages + (t.tile >> c.tiles_log2));
  ok = page >= 0 && page < c.num_pages;
  if (!ok && threadIdx.x % 32 == 0) kv4_bad_page(status, where);
  return ok ? kv4_record(c, page, h, t.tile & ((1 << c.tiles_log2) - 1), d) : 0;
}

// From the codes of the lane's own token to its V word (channels 8 t .. + 3 of
// both tokens of a pair in the even lane, + 4 .. + 7 in the odd), and back.
__device__ __forceinline__ uint32_t swap_pair(uint32_t w, bool odd) {
  const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w : w >> 16, 4);
  return odd ? __byte_perm(got, w, 0x7610) : __byte_perm(w, got, 0x5410);
}

// min and max of packed bf16 pairs; NaN if one of them is
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Codes of 8 values of a group of four lanes' 32, its scale (low half) and minimum (high half).
__device__ __forceinline__ void quantise(const uint4& raw, uint32_t& codes, uint32_t& stat) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t mn = min_bf16x2(min_bf16x2(w[0], w[1]), min_bf16x2(w[2], w[3]));
  uint32_t mx = max_bf16x2(max_bf16x2(w[0], w[1]), max_bf16x2(w[2], w[3]));
  // minimum in the low half, maximum in the high half, both as maxima of (-x, x)
  uint32_t both = max_bf16x2(__byte_perm(mn, mx, 0x5410) ^ 0x8000u, __byte_perm(mn, mx, 0x7632) ^ 0x8000u);
  both = max_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, 1));
  both = max_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, 2));
  // halves, so that max - min cannot overflow
  const float lo = -lo16(both), hi = hi16(both), hlo = -0.5f * lo;
  const float span = fmaf(0.5f, hi, hlo);
  // span / 7.5: the product put right by its remainder, so that a quotient of
  // few bits (one on a bf16 tie has 9) is exact
  constexpr float kInv = 1.0f / 7.5f;
  float s32 = span * kInv;
  s32 = fmaf(fmaf(-s32, 7.5f, span), kInv, s32);
  uint32_t s_bits = pack_bf16x2(s32, 0.0f) & 0xffffu;
  uint32_t lo_bits = __float_as_uint(lo) >> 16;
  codes = 0;
  if (!(fmaxf(fabsf(lo), fabsf(hi)) < INFINITY) || lo != lo || hi != hi) {
    s_bits = 0x7fc0u;
    lo_bits = 0;
  } else if (s_bits < 0x0100u) {  // below 2^-125: held as the minimum
    const uint32_t size = lo_bits & 0x7fffu;
    s_bits = size >= 0x0100u + (13u << 7) ? size - (13u << 7) : 0u;
  } else {
    const float s = 0.5f * __uint_as_float(s_bits << 16);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
    const float2 inv2 = make_float2(inv, inv), s2 = make_float2(-s, -s);
    const float2 up = make_float2(kRound, kRound), down = make_float2(-kRound, -kRound);
    float2 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // values j and j + 4
      const uint32_t u = w[j / 2], v = w[2 + j / 2];
      const float2 x = j % 2 ? make_float2(hi16(u), hi16(v)) : make_float2(lo16(u), lo16(v));
      const float2 d = fma2(x, make_float2(0.5f, 0.5f), make_float2(hlo, hlo));
      const float2 e = mul2(d, inv2);
      q[j] = add2(add2(fma2(fma2(e, s2, d), inv2, e), up), down);  // the quotient, put right as above, rounded
    }
    const float2 k = make_float2(16.0f, 16.0f);
    const float2 all = add2(fma2(fma2(fma2(q[3], k, q[2]), k, q[1]), k, q[0]), up);
    codes = __byte_perm(__float_as_uint(all.x), __float_as_uint(all.y), 0x5410);
  }
  stat = s_bits | lo_bits << 16;
}

// Writes 8 channels' codes of token r, and in one lane of four the group's statistics.
template <int D>
__device__ __forceinline__ void put_token(uint8_t* rec, int isv, int r, int g, int t, uint32_t codes, uint32_t stat) {
  constexpr int G = D / 32;
  const int r8 = r % 8, up = r / 8, at = (r8 * G + g) * 4 + up * 2;
  if (isv) {
    uint8_t* const v = rec + 8 * D + ((g * 8 + 2 * t) * 4 + r8 / 2) * 8 + up * 4 + r8 % 2 * 2;
    *reinterpret_cast<uint16_t*>(v) = (uint16_t)codes;
    *reinterpret_cast<uint16_t*>(v + 32) = (uint16_t)(codes >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(rec + ((g * 8 + r8) * 4 + t) * 8 + up * 4) = codes;
  }
  if (t == g % 4) {
    *reinterpret_cast<uint16_t*>(rec + (isv ? 18 : 16) * D + at) = (uint16_t)stat;
    *reinterpret_cast<uint16_t*>(rec + (isv ? 19 * D + (g * 16 + r) * 2 : 17 * D + at)) = (uint16_t)(stat >> 16);
  }
}

// The item (the block's: the same for all its warps), head and side (0 keys, 1
// values) of a warp. False where it has nothing to do.
__device__ __forceinline__ bool warp_item(const Kv4Pool& c, Kv4Item& it, int& h, int& isv) {
  const int w = blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32;
  it = kv4_item(c, (int)blockIdx.x);
  isv = w >= c.Hkv;
  h = w - (isv ? c.Hkv : 0);
  return h < c.Hkv && it.begin < it.end;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_tiles_kernel(const __grid_constant__ AppendParams p) {
  constexpr int G = D / 32;
  Kv4Item it;
  int h, isv;
  if (!warp_item(p.c, it, h, isv) || it.tile < 0) return;
  bool ok;
  uint8_t* const rec = p.pool + record_at(p.c, it, h, D, p.status, 0x510, ok);
  if (!ok) return;
  const int lane = threadIdx.x % 32, r = lane / 4, t = lane % 4;
  const bool odd = r & 1;
  const int tok = it.tile * kKv4Tile + r;
  const bool has[2] = {tok >= it.begin && tok < it.end, tok + 8 >= it.begin && tok + 8 < it.end};
  const bool full = it.end - it.begin == kKv4Tile;
  const long long ts = isv ? p.ts[1] : p.ts[0];
  const uint16_t* const x = (isv ? p.x[1] : p.x[0]) + (long long)(it.first + tok) * ts + h * (isv ? p.hs[1] : p.hs[0]) + 8 * t;
  uint4 raw[2][G];
#pragma unroll
  for (int up = 0; up < 2; ++up)
#pragma unroll
    for (int g = 0; g < G; ++g)
      raw[up][g] = has[up] ? __ldcs(reinterpret_cast<const uint4*>(x + 8 * up * ts + 32 * g)) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint32_t codes[2], stat[2];
    quantise(raw[0][g], codes[0], stat[0]);
    quantise(raw[1][g], codes[1], stat[1]);
    const int at = (r * G + g) * 4;  // of the two tokens' statistics
    if (full) {
      if (isv) {
        codes[0] = swap_pair(codes[0], odd);
        codes[1] = swap_pair(codes[1], odd);
      }
      const int word = isv ? 8 * D + ((g * 8 + 2 * t + odd) * 4 + r / 2) * 8 : (g * 32 + lane) * 8;
      *reinterpret_cast<uint2*>(rec + word) = make_uint2(codes[0], codes[1]);
      if (t == g % 4) {
        *reinterpret_cast<uint32_t*>(rec + (isv ? 18 : 16) * D + at) = __byte_perm(stat[0], stat[1], 0x5410);
        const uint32_t lo = __byte_perm(stat[0], stat[1], 0x7632);
        if (isv) {
          *reinterpret_cast<uint16_t*>(rec + 19 * D + (g * 16 + r) * 2) = (uint16_t)lo;
          *reinterpret_cast<uint16_t*>(rec + 19 * D + (g * 16 + r + 8) * 2) = (uint16_t)(lo >> 16);
        } else {
          *reinterpret_cast<uint32_t*>(rec + 17 * D + at) = lo;
        }
      }
    } else {  // the other tokens of the record stay as they are
#pragma unroll
      for (int up = 0; up < 2; ++up)
        if (has[up]) put_token<D>(rec, isv, r + 8 * up, g, t, codes[up], stat[up]);
    }
  }
}

// One thread holds 8 channels of one token, head and side; four lanes a group.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_rows_kernel(const __grid_constant__ AppendParams p) {
  constexpr int C = D / 8;  // chunks of a row
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int chunk = (int)(item % C);
  const int isv = (int)(item / C % 2);
  const int h = (int)(item / (2 * C) % p.c.Hkv);
  const long long row = item / (2 * C) / p.c.Hkv;
  uint8_t* rec = nullptr;
  int r = 0;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (row < p.c.total) {
    const int b = kv4_seq_of(p.c, (int)row);
    int first, n;
    kv4_rows(p.c, b, first, n);
    const int i = (int)row - first;
    const int pos = kv4_len(p.c, b) - n + i;
    if (b < p.c.num_seqs && i >= 0 && i < n && pos >= 0) {
      const int tile = pos / kKv4Tile;
      const int page = __ldg(p.c.table + (size_t)b * p.c.max_pages + (tile >> p.c.tiles_log2));
      if (page >= 0 && page < p.c.num_pages) {
        rec = p.pool + kv4_record(p.c, page, h, tile & ((1 << p.c.tiles_log2) - 1), D);
        r = pos % kKv4Tile;
        raw = __ldcs(reinterpret_cast<const uint4*>(p.x[isv] + row * p.ts[isv] + h * p.hs[isv] + 8 * chunk));
      } else if (chunk == 0) {
        kv4_bad_page(p.status, 0x510);
      }
    }
  }
  uint32_t codes, stat;
  quantise(raw, codes, stat);
  if (rec != nullptr) put_token<D>(rec, isv, r, chunk / 4, chunk % 4, codes, stat);
}

struct GatherParams {
  Kv4Pool c;
  uint16_t* y[2];  // k, v: bf16 [total, Hkv, d]
  int* status;
};

// The values of 8 codes as bf16.
__device__ __forceinline__ uint4 dequantise(uint32_t codes, float s, float m) {
  // a code 4 j bits up in the mantissa of 2^23 is 2^23 + 16^j code: no shifts
  // but one for the upper four; the scale takes the 16^j back
  const float2 s01 = make_float2(s, s * 0.0625f), s23 = mul2(s01, make_float2(0.00390625f, 0.00390625f));
  const float2 m2 = make_float2(m, m), k = make_float2(-8388608.0f, -8388608.0f);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? codes >> 16 : codes;
    const float2 a = make_float2(__uint_as_float((w & 0xfu) | 0x4b000000u), __uint_as_float((w & 0xf0u) | 0x4b000000u));
    const float2 b = make_float2(__uint_as_float((w & 0xf00u) | 0x4b000000u), __uint_as_float((w & 0xf000u) | 0x4b000000u));
    const float2 x = fma2(add2(a, k), s01, m2), y = fma2(add2(b, k), s23, m2);
    out[2 * i] = pack_bf16x2(x.x, x.y);
    out[2 * i + 1] = pack_bf16x2(y.x, y.y);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_tiles_kernel(const __grid_constant__ GatherParams p) {
  constexpr int G = D / 32;
  Kv4Item it;
  int h, isv;
  if (!warp_item(p.c, it, h, isv)) return;
  bool ok = false;  // tokens below 0 and on no page of the pool are 0
  const uint8_t* const rec = p.c.data + (it.tile < 0 ? 0 : record_at(p.c, it, h, D, p.status, 0x520, ok));
  const int lane = threadIdx.x % 32, r = lane / 4, t = lane % 4;
  const bool odd = r & 1;
  const int tok = it.tile * kKv4Tile + r;
  const bool has[2] = {tok >= it.begin && tok < it.end, tok + 8 >= it.begin && tok + 8 < it.end};
  uint2 word[G];
  uint32_t sc[G], lo[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    word[g] = make_uint2(0, 0);
    sc[g] = lo[g] = 0;
    if (ok) {
      const int at = isv ? 8 * D + ((g * 8 + 2 * t + odd) * 4 + r / 2) * 8 : (g * 32 + lane) * 8;
      word[g] = __ldg(reinterpret_cast<const uint2*>(rec + at));
      sc[g] = __ldg(reinterpret_cast<const uint32_t*>(rec + (isv ? 18 : 16) * D + (r * G + g) * 4));
      if (isv)
        lo[g] = __byte_perm(__ldg(reinterpret_cast<const uint16_t*>(rec + 19 * D + (g * 16 + r) * 2)),
                            __ldg(reinterpret_cast<const uint16_t*>(rec + 19 * D + (g * 16 + r + 8) * 2)), 0x5410);
      else
        lo[g] = __ldg(reinterpret_cast<const uint32_t*>(rec + 17 * D + (r * G + g) * 4));
    }
  }
  uint16_t* const y = (isv ? p.y[1] : p.y[0]) + ((long long)(it.first + tok) * p.c.Hkv + h) * D + 8 * t;
  const long long eight = 8LL * p.c.Hkv * D;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (isv) {
      word[g].x = swap_pair(word[g].x, odd);
      word[g].y = swap_pair(word[g].y, odd);
    }
    const uint4 a = dequantise(word[g].x, lo16(sc[g]), lo16(lo[g])), b = dequantise(word[g].y, hi16(sc[g]), hi16(lo[g]));
    if (has[0]) __stcs(reinterpret_cast<uint4*>(y + 32 * g), a);
    if (has[1]) __stcs(reinterpret_cast<uint4*>(y + eight + 32 * g), b);
  }
}

// One thread writes 8 channels of one token, head and side.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_rows_kernel(const __grid_constant__ GatherParams p) {
  constexpr int G = D / 32, C = D / 8;
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int chunk = (int)(item % C);
  const int isv = (int)(item / C % 2);
  const int h = (int)(item / (2 * C) % p.c.Hkv);
  const long long row = item / (2 * C) / p.c.Hkv;
  if (row >= p.c.total) return;
  const int b = kv4_seq_of(p.c, (int)row);
  int first, n;
  kv4_rows(p.c, b, first, n);
  const int i = (int)row - first;
  if (i < 0 || i >= n) return;
  const int pos = kv4_len(p.c, b) - n + i;
  uint4 out = make_uint4(0, 0, 0, 0);
  if (pos >= 0) {
    const int tile = pos / kKv4Tile, r = pos % kKv4Tile;
    const int page = __ldg(p.c.table + (size_t)b * p.c.max_pages + (tile >> p.c.tiles_log2));
    if (page >= 0 && page < p.c.num_pages) {
      const uint8_t* const rec = p.c.data + kv4_record(p.c, page, h, tile & ((1 << p.c.tiles_log2) - 1), D);
      const int g = chunk / 4, t = chunk % 4, r8 = r % 8, up = r / 8;
      const int at = (r8 * G + g) * 4 + up * 2;
      uint32_t codes, s_bits, lo_bits;
      if (!isv) {
        codes = *reinterpret_cast<const uint32_t*>(rec + ((g * 8 + r8) * 4 + t) * 8 + up * 4);
        s_bits = *reinterpret_cast<const uint16_t*>(rec + 16 * D + at);
        lo_bits = *reinterpret_cast<const uint16_t*>(rec + 17 * D + at);
      } else {
        const uint8_t* const v = rec + 8 * D + ((g * 8 + 2 * t) * 4 + r8 / 2) * 8 + up * 4 + r8 % 2 * 2;
        codes = *reinterpret_cast<const uint16_t*>(v) | (uint32_t)*reinterpret_cast<const uint16_t*>(v + 32) << 16;
        s_bits = *reinterpret_cast<const uint16_t*>(rec + 18 * D + at);
        lo_bits = *reinterpret_cast<const uint16_t*>(rec + 19 * D + (g * 16 + r) * 2);
      }
      out = dequantise(codes, lo16(s_bits), lo16(lo_bits));
    } else if (chunk == 0) {
      kv4_bad_page(p.status, 0x520);
    }
  }
  __stcs(reinterpret_cast<uint4*>(p.y[isv] + (row * p.c.Hkv + h) * D + 8 * chunk), out);
}

// Page copies: 16 KiB a block.
constexpr int kCopyVectors = 4;
__global__ void __launch_bounds__(kThreads) kv4_copy_kernel(uint8_t* pool, size_t layer_bytes, size_t page_bytes,
                                                            int num_pages, const int* __restrict__ src,
                                                            const int* __restrict__ dst, int chunks, int* status) {
  const int pair = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int from = __ldg(src + pair), to = __ldg(dst + pair);
  if (from < 0 || from >= num_pages || to < 0 || to >= num_pages) {
    if (threadIdx.x == 0) kv4_bad_page(status, 0x530);
    return;
  }
  if (from == to) return;
  uint8_t* const layer = pool + blockIdx.y * layer_bytes;
  const uint4* const a = reinterpret_cast<const uint4*>(layer + from * page_bytes);
  uint4* const z = reinterpret_cast<uint4*>(layer + to * page_bytes);
  const size_t n = page_bytes / 16, at = (size_t)chunk * kThreads * kCopyVectors + threadIdx.x;
  uint4 v[kCopyVectors];
#pragma unroll
  for (int i = 0; i < kCopyVectors; ++i)
    if (at + i * kThreads < n) v[i] = __ldcs(a + at + i * kThreads);
#pragma unroll
  for (int i = 0; i < kCopyVectors; ++i)
    if (at + i * kThreads < n) __stcs(z + at + i * kThreads, v[i]);
}

// Whole records, a warp each, where a sequence has kTileRows rows or more on
// average; single rows below that, where most of a record's lanes would have
// nothing to do. Append and gather of n rows in each of 256 sequences, rows /
// records (us): n = 1 12 / 20, 8 22 / 29, 16 33 / 33, 32 55 / 45; of one
// sequence: 16 10 / 14, 32 12 / 14.
constexpr int kTileRows = 32;
bool by_tiles(const Kv4Pool& c) { return (long long)c.total >= (long long)kTileRows * c.num_seqs; }

struct CacheGrid {
  dim3 grid;
  int threads;  // 0: too much for a launch
};
CacheGrid cache_grid(const Kv4Pool& c, int d) {
  CacheGrid g;
  long long x;
  unsigned y = 1;
  if (by_tiles(c)) {
    const int warps = std::min(kThreads / 32, 2 * c.Hkv);
    g.threads = 32 * warps;
    x = kv4_num_items(c);
    y = (2u * c.Hkv + warps - 1) / warps;
  } else {
    g.threads = kThreads;
    x = ((long long)c.total * c.Hkv * 2 * (d / 8) + kThreads - 1) / kThreads;
  }
  if (x > 0x7fffffffLL) g.threads = 0;
  g.grid = dim3((unsigned)x, y);
  return g;
}

template <typename F>
void by_dim(int d, F f) {
  if (d == 64) f(std::integral_constant<int, 64>());
  else if (d == 96) f(std::integral_constant<int, 96>());
  else if (d == 128) f(std::integral_constant<int, 128>());
  else f(std::integral_constant<int, 256>());
}

}  // namespace

attn_status_t kv4_pool_params(Kv4Pool* c, const void* pool, const int* page_table, const int* seq_lens, const int* cu,
                              int num_seqs, int max_pages, int num_pages, int page_size, int total, int Hkv, int d) {
  if (!pool || !page_table || !seq_lens) return ATTN_ERR_INVALID_ARG;
  if (num_seqs <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0 || total <= 0 || Hkv <= 0 || d <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (!cu && total % num_seqs) return ATTN_ERR_INVALID_ARG;
  if (page_size < kKv4Tile || page_size > 1024 || (page_size & (page_size - 1))) return ATTN_ERR_UNSUPPORTED;
  if (d != 64 && d != 96 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || Hkv > 65535 || (long long)max_pages * page_size > kKv4MaxTokens) return ATTN_ERR_UNSUPPORTED;
  const uintptr_t ints = reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(seq_lens) |
                         reinterpret_cast<uintptr_t>(cu);
  if ((reinterpret_cast<uintptr_t>(pool) & 15u) || (ints & 3u)) return ATTN_ERR_ALIGNMENT;
  c->data = static_cast<const uint8_t*>(pool);
  c->table = page_table;
  c->seq_lens = seq_lens;
  c->cu = cu;
  c->rows_per_seq = cu ? 0 : total / num_seqs;
  c->num_seqs = num_seqs;
  c->max_pages = max_pages;
  c->num_pages = num_pages;
  c->Hkv = Hkv;
  c->tiles_log2 = 0;
  while ((kKv4Tile << c->tiles_log2) < page_size) ++c->tiles_log2;
  c->total = total;
  return ATTN_OK;
}

}  // namespace attn_sm100

using namespace attn_sm100;

extern "C" {

size_t attn_kv4_page_bytes(int Hkv, int d, int page_size) {
  if (Hkv <= 0 || page_size < kKv4Tile || page_size > 1024 || (page_size & (page_size - 1)) ||
      (d != 64 && d != 96 && d != 128 && d != 256))
    return 0;
  return (size_t)Hkv * (page_size / kKv4Tile) * kv4_record_bytes(d);
}

attn_status_t attn_kv4_append(const void* k, const void* v, long long k_token_stride, long long k_head_stride,
                              long long v_token_stride, long long v_head_stride, void* pool, const int* page_table,
                              const int* seq_lens, const int* cu_seqlens, int num_seqs, int max_pages, int num_pages,
                              int page_size, int total, int Hkv, int d, void* stream) {
  if (!k || !v) return ATTN_ERR_INVALID_ARG;
  AppendParams p;
  const attn_status_t s = kv4_pool_params(&p.c, pool, page_table, seq_lens, cu_seqlens, num_seqs, max_pages, num_pages,
                                          page_size, total, Hkv, d);
  if (s != ATTN_OK) return s;
  if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0) return ATTN_ERR_INVALID_ARG;
  if ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) % 8 ||
      ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u))
    return ATTN_ERR_ALIGNMENT;
  const CacheGrid g = cache_grid(p.c, d);
  if (g.threads == 0) return ATTN_ERR_UNSUPPORTED;
  p.status = device_status_word();
  if (!p.status) return ATTN_ERR_CUDA;
  p.pool = static_cast<uint8_t*>(pool);
  p.x[0] = static_cast<const uint16_t*>(k);
  p.x[1] = static_cast<const uint16_t*>(v);
  p.ts[0] = k_token_stride;
  p.ts[1] = v_token_stride;
  p.hs[0] = k_head_stride;
  p.hs[1] = v_head_stride;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_dim(d, [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (by_tiles(p.c)) kv4_append_tiles_kernel<D><<<g.grid, g.threads, 0, st>>>(p);
    else kv4_append_rows_kernel<D><<<g.grid, g.threads, 0, st>>>(p);
  });
  return cuda_error_status(cudaGetLastError());
}

attn_status_t attn_kv4_gather(const void* pool, const int* page_table, const int* seq_lens, const int* cu_seqlens,
                              int num_seqs, int max_pages, int num_pages, int page_size, int total, int Hkv, int d,
                              void* k, void* v, void* stream) {
  if (!k || !v) return ATTN_ERR_INVALID_ARG;
  GatherParams p;
  const attn_status_t s = kv4_pool_params(&p.c, pool, page_table, seq_lens, cu_seqlens, num_seqs, max_pages, num_pages,
                                          page_size, total, Hkv, d);
  if (s != ATTN_OK) return s;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) return ATTN_ERR_ALIGNMENT;
  const CacheGrid g = cache_grid(p.c, d);
  if (g.threads == 0) return ATTN_ERR_UNSUPPORTED;
  if (k == v) return ATTN_ERR_INVALID_ARG;
  p.status = device_status_word();
  if (!p.status) return ATTN_ERR_CUDA;
  p.y[0] = static_cast<uint16_t*>(k);
  p.y[1] = static_cast<uint16_t*>(v);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_dim(d, [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (by_tiles(p.c)) kv4_gather_tiles_kernel<D><<<g.grid, g.threads, 0, st>>>(p);
    else kv4_gather_rows_kernel<D><<<g.grid, g.threads, 0, st>>>(p);
  });
  return cuda_error_status(cudaGetLastError());
}

attn_status_t attn_kv4_copy_pages(void* pool, int num_layers, int num_pages, size_t page_bytes, const int* src,
                                  const int* dst, int num_pairs, void* stream) {
  if (!pool || !src || !dst || num_layers <= 0 || num_pages <= 0 || page_bytes == 0 || num_pairs <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (page_bytes % 16 || (reinterpret_cast<uintptr_t>(pool) & 15u) ||
      ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 3u))
    return ATTN_ERR_ALIGNMENT;
  const size_t block_bytes = (size_t)kThreads * kCopyVectors * 16;
  const size_t chunks = (page_bytes + block_bytes - 1) / block_bytes;
  if (num_layers > 65535 || chunks > 0x7fffffffULL || chunks * (size_t)num_pairs > 0x7fffffffULL)
    return ATTN_ERR_UNSUPPORTED;
  int* const status = device_status_word();
  if (!status) return ATTN_ERR_CUDA;
  kv4_copy_kernel<<<dim3((unsigned)(chunks * num_pairs), num_layers), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint8_t*>(pool), (size_t)num_pages * page_bytes, page_bytes, num_pages, src, dst, (int)chunks, status);
  return cuda_error_status(cudaGetLastError());
}

}  // extern "C"
