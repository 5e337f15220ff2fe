// kv4_format.cuh — the 4-bit key/value cache's records and its page table, as
// the kernels read them.
//
// A record holds 16 tokens of one kv head in 20 d bytes, G = d / 32 groups of
// 32 channels; each token and group has a bf16 minimum and a bf16 scale:
//     value = minimum + scale * code,  code = 0 .. 15.
//   K codes  at 0      words [G][8 r][4 t][2 hi]: token r + 8 hi, channel
//                      32 g + 8 t + n in bits 4 n .. 4 n + 3
//   V codes  at 8 d    words [G][8 a][4 t][2 hi]: tokens 2 t + 8 hi + p,
//                      channel 32 g + 4 a + n in bits 16 p + 4 n ..
//   K scale  at 16 d   bf16 [8 r][G][2 hi], token r + 8 hi
//   K min    at 17 d   the same
//   V scale  at 18 d   the same
//   V min    at 19 d   bf16 [G][16 tokens]
// The words are the operands of the 16 x 8 x 16 matrix instruction as its
// lanes hold them: lane 4 r + t reads its keys r and r + 8 of one K group as 8
// consecutive bytes, and a nibble in the low bits of a 16-bit half is the fp16
// subnormal code * 2^-24, so `word & 0x000f000f` is an operand register and
// `word & 0x00f000f0` one scaled by 16 (attn_kv4_sm100.cu).
//
// pool: uint8 [num_pages][Hkv][page_size / 16][20 d]. Token j of sequence b is
// in page table[b][j / page_size].
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/attn.h"

namespace attn_sm100 {

constexpr int kKv4Tile = 16;  // tokens of a record
// Most tokens that a page table may hold: positions, and a few records' worth
// behind the last one, are computed in 32 bits.
constexpr int kKv4MaxTokens = 0x7fff0000;

__host__ __device__ constexpr int kv4_record_bytes(int d) { return 20 * d; }

struct Kv4Pool {
  const uint8_t* data;
  const int* table;      // [num_seqs][max_pages]
  const int* seq_lens;   // [num_seqs] tokens in the cache
  const int* cu;         // [num_seqs + 1] row offsets of the call's tokens, or null:
  int rows_per_seq;      //   every sequence has this many
  int num_seqs, max_pages, num_pages;
  int Hkv;
  int tiles_log2;        // log2(page_size / 16)
  int total;             // rows of the call (tokens over all sequences)
};

// Tokens of sequence b in the cache, clamped to what its table row can hold.
__device__ __forceinline__ int kv4_len(const Kv4Pool& c, int b) {
  return min(max(__ldg(c.seq_lens + b), 0), c.max_pages << (c.tiles_log2 + 4));
}

// First row and number of rows of sequence b, clamped to [0, total].
__device__ __forceinline__ void kv4_rows(const Kv4Pool& c, int b, int& first, int& n) {
  if (c.cu == nullptr) {
    first = b * c.rows_per_seq;
    n = c.rows_per_seq;
  } else {
    first = min(max(__ldg(c.cu + b), 0), c.total);
    n = max(min(__ldg(c.cu + b + 1), c.total) - first, 0);
  }
}

// Tiles of 16 tokens that the call's rows lie in. A sequence's n rows touch at
// most n / 16 + 2 of them, so with the sequences' first rows off[s] the items
// v(s) = off[s] / 16 + 2 s onwards are its own, and total / 16 + 2 num_seqs
// items hold them all (rows_per_seq: as many items for each, counted exactly).
__host__ __device__ __forceinline__ int kv4_items_per_seq(int rows) { return (rows + kKv4Tile - 2) / kKv4Tile + 1; }

__host__ __device__ __forceinline__ long long kv4_num_items(const Kv4Pool& c) {
  return c.cu == nullptr ? (long long)c.num_seqs * kv4_items_per_seq(c.rows_per_seq)
                         : c.total / kKv4Tile + 2LL * c.num_seqs;
}

// One item: the tokens tile * 16 .. + 15 of sequence b, of which the call's are
// [begin, end) (from token 0 on; possibly none), token j being row first + j.
struct Kv4Item {
  int b, tile, begin, end, first;
};

__device__ __forceinline__ Kv4Item kv4_item(const Kv4Pool& c, int i) {
  Kv4Item t;
  int nth;
  if (c.cu == nullptr) {
    const int per = kv4_items_per_seq(c.rows_per_seq);
    t.b = i / per;
    nth = i - t.b * per;
  } else {
    int lo = 0, hi = c.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (min(max(__ldg(c.cu + mid), 0), c.total) / kKv4Tile + 2 * mid <= i) lo = mid;
      else hi = mid - 1;
    }
    t.b = lo;
    nth = i - (min(max(__ldg(c.cu + lo), 0), c.total) / kKv4Tile + 2 * lo);
  }
  int row, n;
  kv4_rows(c, t.b, row, n);
  const int end = kv4_len(c, t.b), begin = end - n;
  t.tile = (begin >> 4) + nth;  // tokens below 0 are in tiles below 0
  t.begin = max(begin, t.tile * kKv4Tile);
  t.end = min(end, t.tile * kKv4Tile + kKv4Tile);
  t.first = row - begin;
  return t;
}

// The sequence that owns row i: the largest b whose rows begin at or before i.
__device__ __forceinline__ int kv4_seq_of(const Kv4Pool& c, int i) {
  if (c.cu == nullptr) return i / c.rows_per_seq;
  int lo = 0, hi = c.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(c.cu + mid) <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Byte offset in the pool of the record of (page, head h, tile of the page).
__device__ __forceinline__ size_t kv4_record(const Kv4Pool& c, int page, int h, int tile, int d) {
  return ((((size_t)page * c.Hkv + h) << c.tiles_log2) + tile) * (size_t)kv4_record_bytes(d);
}

// Records a page id outside the pool in the device status word, if it is the first failure there.
__device__ __forceinline__ void kv4_bad_page(int* status, int where) {
  if (atomicCAS(status, 0, ATTN_ERR_INVALID_ARG) == 0) status[1] = where;
}

}  // namespace attn_sm100
