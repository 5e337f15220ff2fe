// kv4_cache_sm100.cu — writing, reading back and copying pages of the 4-bit
// key/value cache (records and page table: kv4_format.cuh).
//
// Quantisation, for a token, kv head and group of 32 channels x_c (bf16):
//   lo = min_c x_c (a bf16 number itself, so exact), s = bf16((max - lo) / 15),
//   code_c = min(round((x_c - lo) / s), 15), ties to even; the cache then
//   stands for lo + s * code_c, off by at most s / 2 + 15 * 2^-9 s.
// A group whose spread is below 15 * 2^-126 is held as its minimum (s = 0). A
// group with a NaN or an infinity is held as NaN (s = NaN, lo = 0).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "attn_internal.h"
#include "kv4_format.cuh"
#include "sm100_ptx.cuh"

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

// One thread holds 8 channels of one token, head and K or V; four lanes a group.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int G = D / 32, C = D / 8;  // chunks of a row
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int chunk = (int)(item % C);
  const int isv = (int)(item / C % 2);
  const int h = (int)(item / (2 * C) % p.c.Hkv);
  const long long tok = item / (2 * C) / p.c.Hkv;
  uint8_t* rec = nullptr;
  int r = 0;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (tok < p.c.total) {
    const int b = kv4_seq_of(p.c, (int)tok);
    int first, n;
    kv4_rows(p.c, b, first, n);
    const int i = (int)tok - first;
    const int pos = kv4_len(p.c, b) - n + i;
    if (b < p.c.num_seqs && i >= 0 && i < n && pos >= 0) {
      const int tile = pos / kKv4Tile;
      const int page = __ldg(p.c.table + (size_t)b * p.c.max_pages + (tile >> p.c.tiles_log2));
      if (page >= 0 && page < p.c.num_pages) {
        rec = p.pool + kv4_record(p.c, page, h, tile & ((1 << p.c.tiles_log2) - 1), D);
        r = pos % kKv4Tile;
        raw = __ldcs(reinterpret_cast<const uint4*>(p.x[isv] + tok * p.ts[isv] + h * p.hs[isv] + 8 * chunk));
      } else if (chunk == 0) {
        kv4_bad_page(p.status, 0x510);
      }
    }
  }
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  // halves, so that max - min cannot overflow; exact but for subnormals
  float x[8], lo = INFINITY, hi = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t bits = i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16;
    bad |= (bits & 0x7f800000u) == 0x7f800000u;
    x[i] = __uint_as_float(bits);
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
  }
  if (rec == nullptr) return;
  uint32_t s_bits = pack_bf16x2((0.5f * hi - 0.5f * lo) / 7.5f, 0.0f) & 0xffffu;
  uint32_t lo_bits = __float_as_uint(lo) >> 16;
  if (s_bits < 0x0080u) s_bits = 0;  // below 2^-126
  if (bad) {
    s_bits = 0x7fc0u;
    lo_bits = 0;
  }
  uint32_t codes = 0;
  if (s_bits != 0 && !bad) {
    const float s = 0.5f * __uint_as_float(s_bits << 16), inv = 1.0f / s, half = 0.5f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = 0.5f * x[i] - 0.5f * lo;
      // the quotient through the reciprocal, put right by the exact remainder
      float q = rintf(d * inv);
      const float rem = fmaf(-q, s, d);
      const bool odd = ((int)q & 1) != 0;
      if (rem > half || (rem == half && odd)) q += 1.0f;
      else if (rem < -half || (rem == -half && odd)) q -= 1.0f;
      codes |= (uint32_t)min(max((int)q, 0), 15) << (4 * i);
    }
  }
  const int gr = chunk / 4, t = chunk % 4, r8 = r % 8, up = r / 8;
  const int stat = (r8 * G + gr) * 4 + up * 2;
  if (!isv) {
    *reinterpret_cast<uint32_t*>(rec + ((gr * 8 + r8) * 4 + t) * 8 + up * 4) = codes;
    if (t == 0) {
      *reinterpret_cast<uint16_t*>(rec + 16 * D + stat) = (uint16_t)s_bits;
      *reinterpret_cast<uint16_t*>(rec + 17 * D + stat) = (uint16_t)lo_bits;
    }
  } else {
    uint8_t* const v = rec + 8 * D + ((gr * 8 + 2 * t) * 4 + r8 / 2) * 8 + up * 4 + (r % 2) * 2;
    *reinterpret_cast<uint16_t*>(v) = (uint16_t)codes;
    *reinterpret_cast<uint16_t*>(v + 32) = (uint16_t)(codes >> 16);
    if (t == 0) {
      *reinterpret_cast<uint16_t*>(rec + 18 * D + stat) = (uint16_t)s_bits;
      *reinterpret_cast<uint16_t*>(rec + 19 * D + (gr * 16 + r) * 2) = (uint16_t)lo_bits;
    }
  }
}

struct GatherParams {
  Kv4Pool c;
  uint16_t* y[2];  // k, v: bf16 [total, Hkv, d]
  int* status;
};

// One thread writes 8 channels of one token, head and K or V.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int G = D / 32, C = D / 8;
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int chunk = (int)(item % C);
  const int isv = (int)(item / C % 2);
  const int h = (int)(item / (2 * C) % p.c.Hkv);
  const long long tok = item / (2 * C) / p.c.Hkv;
  if (tok >= p.c.total) return;
  const int b = kv4_seq_of(p.c, (int)tok);
  int first, n;
  kv4_rows(p.c, b, first, n);
  const int i = (int)tok - first;
  if (i < 0 || i >= n) return;
  const int pos = kv4_len(p.c, b) - n + i;
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 0.0f;
  if (pos >= 0) {
    const int tile = pos / kKv4Tile, r = pos % kKv4Tile;
    const int page = __ldg(p.c.table + (size_t)b * p.c.max_pages + (tile >> p.c.tiles_log2));
    if (page >= 0 && page < p.c.num_pages) {
      const uint8_t* const rec = p.c.data + kv4_record(p.c, page, h, tile & ((1 << p.c.tiles_log2) - 1), D);
      const int gr = chunk / 4, t = chunk % 4, r8 = r % 8, up = r / 8;
      const int stat = (r8 * G + gr) * 4 + up * 2;
      uint32_t codes, s_bits, lo_bits;
      if (!isv) {
        codes = *reinterpret_cast<const uint32_t*>(rec + ((gr * 8 + r8) * 4 + t) * 8 + up * 4);
        s_bits = *reinterpret_cast<const uint16_t*>(rec + 16 * D + stat);
        lo_bits = *reinterpret_cast<const uint16_t*>(rec + 17 * D + stat);
      } else {
        const uint8_t* const v = rec + 8 * D + ((gr * 8 + 2 * t) * 4 + r8 / 2) * 8 + up * 4 + (r % 2) * 2;
        codes = *reinterpret_cast<const uint16_t*>(v) | (uint32_t)*reinterpret_cast<const uint16_t*>(v + 32) << 16;
        s_bits = *reinterpret_cast<const uint16_t*>(rec + 18 * D + stat);
        lo_bits = *reinterpret_cast<const uint16_t*>(rec + 19 * D + (gr * 16 + r) * 2);
      }
      const float s = __uint_as_float(s_bits << 16), lo = __uint_as_float(lo_bits << 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf(s, (float)(codes >> (4 * j) & 15u), lo);
    } else if (chunk == 0) {
      kv4_bad_page(p.status, 0x520);
    }
  }
  const uint4 out = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                               pack_bf16x2(f[6], f[7]));
  *reinterpret_cast<uint4*>(p.y[isv] + (tok * p.c.Hkv + h) * D + 8 * chunk) = out;
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

template <typename F64, typename F96, typename F128, typename F256>
void by_dim(int d, F64 f64, F96 f96, F128 f128, F256 f256) {
  if (d == 64) f64();
  else if (d == 96) f96();
  else if (d == 128) f128();
  else f256();
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
  if (num_seqs > 65535 || Hkv > 65535 || (long long)max_pages * page_size > 0x7ffffff0LL) return ATTN_ERR_UNSUPPORTED;
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
  const long long blocks = ((long long)total * Hkv * 2 * (d / 8) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
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
  const unsigned g = (unsigned)blocks;
  by_dim(d, [&] { kv4_append_kernel<64><<<g, kThreads, 0, st>>>(p); },
         [&] { kv4_append_kernel<96><<<g, kThreads, 0, st>>>(p); },
         [&] { kv4_append_kernel<128><<<g, kThreads, 0, st>>>(p); },
         [&] { kv4_append_kernel<256><<<g, kThreads, 0, st>>>(p); });
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
  const long long blocks = ((long long)total * Hkv * 2 * (d / 8) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  p.status = device_status_word();
  if (!p.status) return ATTN_ERR_CUDA;
  p.y[0] = static_cast<uint16_t*>(k);
  p.y[1] = static_cast<uint16_t*>(v);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned g = (unsigned)blocks;
  by_dim(d, [&] { kv4_gather_kernel<64><<<g, kThreads, 0, st>>>(p); },
         [&] { kv4_gather_kernel<96><<<g, kThreads, 0, st>>>(p); },
         [&] { kv4_gather_kernel<128><<<g, kThreads, 0, st>>>(p); },
         [&] { kv4_gather_kernel<256><<<g, kThreads, 0, st>>>(p); });
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
