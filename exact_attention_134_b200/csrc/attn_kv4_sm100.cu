// attn_kv4_sm100.cu — attention over the paged 4-bit cache (kv4_format.cuh)
// for a few query tokens a sequence, and the merge of its split results.
//
//   S_ij = scale * sum_g (s_jg * sum_{c in g} q_ic code_jc + lo_jg * sum_{c in g} q_ic)
//   O_i  = sum_j p_ij (lo_jg + s_jg code_jc) / sum_j p_ij,  p_ij = 2^(S_ij log2(e) - R_i)
// so the codes themselves are the operands of the matrix instructions and the
// keys and values are never rounded: scale and minimum come in afterwards (K:
// scale on the fp32 sums of a group, minima by one instruction against the
// sums of the query's groups) or before (V: p * s, one operand a group; the
// minima times p by one instruction).
//
// Operands. A code in the low bits of a 16-bit half is the fp16 subnormal
// code * 2^-24, exact in the tensor core, and one 4 bits up is 16 times that:
// a word of 8 codes becomes four operand registers with four masks and a
// subtraction. The scores are taken as S^T = K Q^T (16 keys x 8 query rows an
// instruction) and the output as O^T = V^T P^T: with one token and at most 8
// query heads a kv head, 8 columns hold the rows, where 64 or 128 rows of a
// tcgen05 tile would be filled up with zeros, and operands go from the
// dequantised register straight into the instruction; tcgen05 would need them
// written to shared or tensor memory first, and its accumulators read back for
// the scale of every group. Q is scaled by a power of two a row into fp16's
// range; P^T = p * s is fp16 as well, against a reference that follows the row's
// maximum and the keys' scales: 2^7 <= its largest < 2^15. It is rounded once (by
// 2^-11 at most, by 2^-25 below 2^-14, which is 2^-21 of the largest): a second
// piece would double the output's instructions, and against 64 bits the batch
// below is off by 0.00171 where 0.00165 are the result's own rounding. The minima
// take p in two bf16 pieces (16 bits): they cancel against the codes' part.
//
// Work. A unit is a pair of records of one block of query rows (4, 8 or 16 of a
// kv head); the units of all sequences, kv heads and row blocks form one list,
// cut into equal ranges, one per CTA, whatever the lengths. The four warps of a
// CTA take the units of a segment (the part of one row block in its range) in
// turn, each with its own ring of bulk copies and its own softmax state; they
// are joined in shared memory at the segment's end. A row block within one
// range is written out there; one cut by a range's border leaves fp32 partial
// results, which the merge kernel joins. Short caches are not cut (launch).
//
// What bounds it: 1.25 d bytes a cached token and kv head, and for up to 4 rows
// 520 warp instructions a pair of records at d = 128 (5120 bytes: 222 clocks of
// an SM's share of the memory rate, 888 issue slots). Measured (B200, one query
// row of 32 / 8 heads, launches in a graph): 64 sequences of 4096 .. 8192 tokens
// 96 us, 5.3 TB/s (87 with the arithmetic of the records left out); one of 131072
// 42 us (37). From the first kernel on, 64 sequences: a record a step with minima
// on the FMA pipe 162 us; two records a step and minima by a matrix instruction
// 137; four warps and three CTAs an SM instead of eight and two 125; up to four
// rows against both records at once 112; query operands in shared memory 110;
// the fourth operand by subtraction, weights moved instead of masked 102. Five
// tiles of columns a warp, or a warp a tile on a shared ring, were no faster for
// 40 rows (41 and 53 us against 37 with passes of 16): the
// scales and weights of a row cost more than its share of the codes.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attn_internal.h"
#include "kv4_format.cuh"
#include "sm100_rows.cuh"

namespace attn_sm100 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kNone = -3.0e38f;     // reference of a row that has seen no key
constexpr uint32_t kMinScale = 0x1f80u;  // bf16 2^-64: smaller scales count as that, so p stays below 2^79
constexpr float kRoom = 32768.0f;     // p * s stays below 2^15
constexpr float kHead = 8.0f;         // log2 of p * s at a new reference: 2^7 of room before the next one
constexpr int kPair = 2;              // records of a step
constexpr int kAlwaysWhole = 16;      // pairs (512 tokens) that are one CTA's work in every launch

struct Kv4Params {
  Kv4Pool c;
  const uint16_t* q;   // bf16 [total, Hq, d]
  uint16_t* o;         // bf16 [total, Hq, d]
  float* lse;          // fp32 [Hq, total]
  float* part_o;       // [2 * CTAs][columns][d]: partial sums of a range's first and last row block
  float2* part_rl;     // [2 * CTAs][columns]: their reference and exponential sum
  int4* split;         // [CTAs][2]: what the merge does at the range's first border
  int* status;
  int Hq, group;
  int causal;
  int whole;           // units are whole row blocks: nothing to merge
  int min_units;       // smallest range worth a CTA
  float scale_log2;
  unsigned long long timeout_ns;
};

// CTAs of an SM: four where 128 registers a thread hold the accumulators (64
// sequences of 16384 tokens, 8 kv heads of 64, 4 / 8 rows: 121 / 148 us, with
// three 126 / 156), three where 168 do.
constexpr int kv4_ctas(int d, int cols) {
  return d == 64 && cols <= 8 ? 4 : d <= 128 && d * cols <= 1024 ? 3 : 2;
}

template <int D, int COLS>
struct Kv4Cfg {
  static constexpr int kWarps = 4;
  static constexpr int kCtasPerSm = kv4_ctas(D, COLS);
  static constexpr int kStages = 2;
  static constexpr int kRecord = kv4_record_bytes(D);
  static constexpr int kStage = kPair * kRecord;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoin = kWarps / 2 * COLS * D * 4;     // fp32 O of half the warps
  static constexpr int kRl = 2 * kWarps * COLS * 8;           // (reference, sum), two segments
  // query operands of the segment: [record sets * column tiles][groups][lane] of
  // 16 bytes, of 8 bytes for the minima, and a factor a column
  static constexpr int kTiles = COLS == 4 ? kPair : COLS / 8, kMins = (D / 32 + 3) / 4;
  static constexpr int kQ = kTiles * (D / 32) * 512, kQm = kTiles * kMins * 256;
  static constexpr int kBars = kWarps * kStages * 8;
  static constexpr int kSmemBytes = kRing + kJoin + kRl + kQ + kQm + COLS * 4 + kBars + 16;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %5}, {%7, %8}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16_full(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four code operands of a word of 8 codes (bits 16 p + 4 n): n = 0 .. 3, the
// odd ones 16 times their value. The last is a difference of fp16 numbers, off
// the pipe that all the masks need.
struct Codes {
  uint32_t n[4];
};
__device__ __forceinline__ Codes codes_of(uint32_t w) {
  Codes c;
  c.n[0] = w & 0x000f000fu;
  c.n[1] = w & 0x00f000f0u;
  const uint32_t up = __byte_perm(w, 0u, 0x4341);
  c.n[2] = up & 0x000f000fu;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(c.n[3]) : "r"(up), "r"(c.n[2]));
  return c;
}

// 8 x 8 transposition of 16-bit values over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// N consecutive words of shared memory, in the widest loads their alignment allows.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(addr + 4 * i));
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[i]), "=r"(w[i + 1]) : "r"(addr + 4 * i));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[i]) : "r"(addr + 4 * i));
  }
}

__device__ __forceinline__ void lds_pair(uint32_t& a, uint32_t& b, uint32_t addr) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}

__device__ __forceinline__ uint32_t lds_word(uint32_t addr) {
  uint32_t a;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(addr));
  return a;
}

// Quotients of counts that mostly fit 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// A sequence's part in the list of units: `blocks` row blocks for each kv
// head, `units` for each of those (one per pair of records, or one; one also
// for an empty cache, so that its rows get their result).
struct SeqWork {
  int first, n, len, blocks, pairs, units;
};
template <int COLS>
__device__ __forceinline__ SeqWork seq_work(const Kv4Params& p, int b) {
  SeqWork s;
  kv4_rows(p.c, b, s.first, s.n);
  s.len = kv4_len(p.c, b);
  s.blocks = (int)(((uint32_t)s.n * (uint32_t)p.group + COLS - 1) / COLS);  // rows are below 2^31
  s.pairs = max(1, (s.len + kPair * kKv4Tile - 1) / (kPair * kKv4Tile));
  s.units = p.whole ? 1 : s.pairs;
  return s;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// One segment: the pairs [t0, t1) of row block rb of kv head h of sequence b.
struct Segment {
  int b, h, rb, t0, t1;
  SeqWork s;
};

// Finds the segment of the list that holds unit `u` (the whole warp takes
// part). False if the list ends before it. Every CTA walks over all sequences,
// here and for their total: of 16384 sequences of 32 .. 64 tokens (530 us, one kv
// head) nothing of it shows, of 65535 some 340 of 2463 us.
template <int COLS>
__device__ __forceinline__ bool find_segment(const Kv4Params& p, long long u, Segment& g) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int b0 = 0; b0 < p.c.num_seqs; b0 += 32) {
    long long mine = 0;
    if (b0 + lane < p.c.num_seqs) {
      const SeqWork s = seq_work<COLS>(p, b0 + lane);
      mine = (long long)s.blocks * p.c.Hkv * s.units;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned past = __ballot_sync(kFull, base + incl > u);
    if (past) {
      const int l = __ffs(past) - 1;
      g.b = b0 + l;
      g.s = seq_work<COLS>(p, g.b);
      const long long in = u - base - __shfl_sync(kFull, incl - mine, l);
      const long long which = quotient(in, g.s.units);
      g.t0 = (int)(in - which * g.s.units);
      g.h = (int)quotient(which, g.s.blocks);
      g.rb = (int)(which - (long long)g.h * g.s.blocks);
      return true;
    }
    base += __shfl_sync(kFull, incl, 31);
  }
  return false;
}

// Ends a segment with the range's `left` units, or its row block; returns the units behind it.
__device__ __forceinline__ long long end_segment(const Kv4Params& p, Segment& g, long long left) {
  g.t1 = p.whole ? g.s.pairs : (int)min((long long)g.s.pairs, g.t0 + left);
  return left - (p.whole ? 1 : g.t1 - g.t0);
}

// Steps to the next segment of the list (its start). False at the end.
template <int COLS>
__device__ __forceinline__ bool next_segment(const Kv4Params& p, Segment& g) {
  g.t0 = 0;
  if (++g.rb < g.s.blocks) return true;
  g.rb = 0;
  if (++g.h < p.c.Hkv) return true;
  g.h = 0;
  while (++g.b < p.c.num_seqs) {
    g.s = seq_work<COLS>(p, g.b);
    if (g.s.blocks > 0) return true;
  }
  return false;
}

template <int D, int COLS>
__global__ void __launch_bounds__(Kv4Cfg<D, COLS>::kWarps * 32, Kv4Cfg<D, COLS>::kCtasPerSm)
    attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
  using C = Kv4Cfg<D, COLS>;
  constexpr int W = C::kWarps, S = C::kStages, G = D / 32;
  static_assert(S == 2 && kPair == 2, "two stages of two records");
  // At most four rows: an instruction's columns 0 .. 3 take them against record
  // 0 of a pair, 4 .. 7 the same rows against record 1, so that one set of
  // scores, weights and scales in the lanes stands for both records.
  constexpr bool HALF = COLS == 4;
  constexpr int NT = HALF ? 1 : COLS / 8;  // column tiles
  constexpr int Q = HALF ? kPair : 1;      // sets of query operands, by record
  constexpr int MINS = (G + 3) / 4;  // instructions for the minima of a record
  constexpr int kUnroll = C::kCtasPerSm == 4 ? 1 : 2;  // a pair's records side by side: 2 % where registers last
  extern __shared__ __align__(128) uint8_t smem[];
  float* const join = reinterpret_cast<float*>(smem + C::kRing);
  float2* const rl = reinterpret_cast<float2*>(smem + C::kRing + C::kJoin);
  uint8_t* const q_smem = smem + C::kRing + C::kJoin + C::kRl;
  float* const fac_smem = reinterpret_cast<float*>(q_smem + C::kQ + C::kQm);
  uint8_t* const bar_smem = q_smem + C::kQ + C::kQm + COLS * 4;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(bar_smem + C::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * S * C::kStage;
  const uint32_t bars = smem_addr(bar_smem) + warp * S * 8;
  const uint32_t qs = smem_addr(q_smem) + lane * 16, qms = smem_addr(q_smem + C::kQ) + lane * 8;

  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < S; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbarrier_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's range of the list
  long long total = 0;
  for (int b0 = 0; b0 < p.c.num_seqs; b0 += 32) {
    if (b0 + lane < p.c.num_seqs) {
      const SeqWork s = seq_work<COLS>(p, b0 + lane);
      total += (long long)s.blocks * p.c.Hkv * s.units;
    }
  }
  total = warp_sum(total);
  // equal ranges, the first `more` of them one unit longer
  const long long ctas = max(1LL, min((long long)gridDim.x, quotient(total, p.min_units)));
  const long long each = quotient(total, ctas), more = total - each * ctas;
  const long long begin = each * blockIdx.x + min((long long)blockIdx.x, more);
  const long long end = begin + each + ((long long)blockIdx.x < more ? 1 : 0);
  Segment seg;
  const bool any = blockIdx.x < ctas && begin < end && find_segment<COLS>(p, begin, seg);
  if (!p.whole && threadIdx.x == 0) {
    // a row block cut by this range's first border, and by none before: what the merge joins
    int4 a = make_int4(0, 0, 0, 0), z = a;
    if (any && seg.t0 > 0) {
      const long long u0 = begin - seg.t0, u1 = u0 + seg.s.units - 1, border = more * (each + 1);
      auto cta_of = [&](long long u) {
        return (int)(u < border ? quotient(u, each + 1) : more + quotient(u - border, each));
      };
      const int c0 = cta_of(u0), c1 = cta_of(u1);
      if (c0 + 1 == (int)blockIdx.x) {
        a = make_int4(1, c0, c1, seg.h);
        z = make_int4(seg.rb, seg.s.first, seg.s.n, 0);
      }
    }
    p.split[2 * blockIdx.x] = a;
    p.split[2 * blockIdx.x + 1] = z;
  }
  if (!any) return;

  // ---- the ring: this warp's units, over all segments of the range
  int flying = 0;         // stages on their way
  Segment pf = seg;
  long long pf_left = end - begin;
  auto units = [&](const Segment& g) {  // of this warp in segment g (none of an empty cache)
    return g.s.len > 0 ? max(0, (g.t1 - g.t0 - warp + W - 1) / W) : 0;
  };
  pf_left = end_segment(p, pf, pf_left);
  int pf_k = 0, pf_count = units(pf);  // next unit of the warp in pf (t0 + warp + W * pf_k), and how many
  // of unit (pf_k / 32) * 32 + lane: its records, and the bytes to copy from
  // each (both from the first if they lie side by side)
  const uint8_t *pf_from0 = nullptr, *pf_from1 = nullptr;
  uint32_t pf_bytes0 = 0, pf_bytes1 = 0;
  int pf_stage = 0;
  bool pf_more = true;
  uint32_t pf_bad0 = 0, pf_bad1 = 0;  // of the 32 units: a record on no page of the pool
  uint32_t bad = 0;                   // the same, two bits each, of the stages on their way

  auto issue = [&]() {
    while (pf_k >= pf_count) {
      if (!pf_more) return;
      pf_more = pf_left > 0 && next_segment<COLS>(p, pf);
      if (!pf_more) return;
      pf_left = end_segment(p, pf, pf_left);
      pf_k = 0;
      pf_count = units(pf);
    }
    if ((pf_k & 31) == 0) {
      const int t = kPair * (pf.t0 + warp + W * (pf_k + lane));
      auto record = [&](int t_, uint32_t& bad_) {
        const bool there = pf_k + lane < pf_count && t_ * kKv4Tile < pf.s.len;
        const int page = there ? __ldg(p.c.table + (size_t)pf.b * p.c.max_pages + (t_ >> p.c.tiles_log2)) : -1;
        const bool ok_ = (unsigned)page < (unsigned)p.c.num_pages;
        bad_ = __ballot_sync(kFull, there && !ok_);
        if (there && !ok_) kv4_bad_page(p.status, 0x500);
        return ok_ ? p.c.data + kv4_record(p.c, page, pf.h, t_ & ((1 << p.c.tiles_log2) - 1), D) : nullptr;
      };
      pf_from0 = record(t, pf_bad0);
      pf_from1 = record(t + 1, pf_bad1);
      const bool side = pf_from0 != nullptr && pf_from1 == pf_from0 + C::kRecord;
      pf_bytes0 = side ? C::kStage : pf_from0 ? C::kRecord : 0;
      pf_bytes1 = !side && pf_from1 ? C::kRecord : 0;
    }
    const int at = pf_k & 31;
    if (lane == at) {  // the unit's own lane
      const uint32_t bar = bars + 8 * pf_stage, to = ring + pf_stage * C::kStage;
      mbar_arrive_expect_tx(bar, pf_bytes0 + pf_bytes1);
      if (pf_bytes0) bulk_load(to, pf_from0, pf_bytes0, bar);
      if (pf_bytes1) bulk_load(to + C::kRecord, pf_from1, pf_bytes1, bar);
    }
    if (pf_bad0 | pf_bad1) bad |= ((pf_bad0 >> at & 1u) | (pf_bad1 >> at & 1u) << 1) << (2 * flying);
    pf_stage ^= 1;
    ++pf_k;
    ++flying;
  };
#pragma unroll 1
  for (int i = 0; i < S; ++i) issue();

  long long left = end - begin;
  left = end_segment(p, seg, left);
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  int turn = 0;  // parity of the segment, for rl
  while (true) {
    // ---- query rows of the segment, as operands: a column tile by each warp
    float fac[NT][2];
    int limit[NT][2];  // last key that the lane's two columns see
    for (int nt = warp; nt < NT; nt += W) {
      const int row = seg.rb * COLS + nt * 8 + g8 % COLS;
      const bool live = row < seg.s.n * p.group;
      const int tok = seg.s.first + row / p.group;
      const uint16_t* const src = p.q + ((size_t)tok * p.Hq + seg.h * p.group + row % p.group) * D + 8 * t4;
      uint4 raw[G];
      uint32_t top = 0;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        raw[gr] = live ? __ldg(reinterpret_cast<const uint4*>(src + 32 * gr)) : make_uint4(0, 0, 0, 0);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[gr].x & 0x7fff7fffu, raw[gr].y & 0x7fff7fffu),
                                     __vmaxu2(raw[gr].z & 0x7fff7fffu, raw[gr].w & 0x7fff7fffu)));
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      // the row's largest value into [2^13, 2^14): a sixteenth of it, for the
      // codes that stand 4 bits up, still is a normal number down to 2^-24 of
      // it. Small rows take the largest power there is; large ones stop at
      // 2^-90, so that its inverse times 2^24 stays finite with the scale: from
      // 2^106 on (13 - 105 is -92, where fp16 still holds it) a row gets NaN
      const int want = 13 - ((int)(top >> 7) - 127), k = min(max(want, -90), 127);
      const float up = want < -92 ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(k + 127) << 23);
      float mine = 0.0f, other = 0.0f;  // the sums over groups t4 and t4 + 4
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const uint32_t w[4] = {raw[gr].x, raw[gr].y, raw[gr].z, raw[gr].w};
        float f[8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = (i % 2 ? hi16(w[i / 2]) : lo16(w[i / 2])) * up;
          sum += f[i];
        }
        // codes i and i + 4 share a register; 1, 3, 5, 7 stand 4 bits up
        const uint4 q = make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1] * 0.0625f, f[5] * 0.0625f),
                                   pack_f16x2(f[2], f[6]), pack_f16x2(f[3] * 0.0625f, f[7] * 0.0625f));
#pragma unroll
        for (int i = 0; i < Q; ++i)
          reinterpret_cast<uint4*>(q_smem)[((i * NT + nt) * G + gr) * 32 + lane] =
              HALF && g8 / 4 != i ? make_uint4(0, 0, 0, 0) : q;
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        if (t4 == gr % 4) (gr < 4 ? mine : other) = sum * 5.9604644775390625e-8f;  // 2^-24
      }
#pragma unroll
      for (int m = 0; m < MINS; ++m) {  // three bf16 pieces of each sum
        const float s = m ? other : mine;
        const float h = hi16(__float_as_uint(s)), l = hi16(__float_as_uint(s - h));
        const uint2 q = make_uint2(pack_bf16x2(h, l), pack_bf16x2((s - h) - l, 0.0f));
#pragma unroll
        for (int i = 0; i < Q; ++i)
          reinterpret_cast<uint2*>(q_smem + C::kQ)[((i * NT + nt) * MINS + m) * 32 + lane] =
              HALF && g8 / 4 != i ? make_uint2(0, 0) : q;
      }
      // above 0, for the product with a masked score
      if (t4 == 0 && (!HALF || g8 < 4))
        fac_smem[nt * 8 + g8] = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(24 - k + 127) << 23), 1.17549435e-38f);
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // the lane's columns 2 t4 + j
        const int col = (nt * 8 + 2 * t4 + j) % COLS, r = seg.rb * COLS + col;
        fac[nt][j] = fac_smem[col];
        limit[nt][j] = p.causal ? seg.s.len - seg.s.n + min(r / p.group, seg.s.n - 1) : seg.s.len - 1;
      }
    // every key up to this one is seen by all rows of the block
    const int all_see = p.causal ? seg.s.len - seg.s.n + seg.rb * COLS / p.group : seg.s.len - 1;

    float o[NT][2 * G][4], omin[NT][4], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int m = 0; m < 2 * G; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][m][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) omin[nt][i] = 0.0f;
      ref[nt][0] = ref[nt][1] = kNone;
      sum[nt][0] = sum[nt][1] = 0.0f;
    }

    const int mine = units(seg);
    int key = (seg.t0 + warp) * kPair * kKv4Tile + g8;  // the lane's keys: key + 8 i
#pragma unroll 1
    for (int k = 0; k < mine; ++k, key += W * kPair * kKv4Tile) {
      ok = ok && __all_sync(kFull, bounded_wait(bars + 8 * stage, phase, abort_flag, p.timeout_ns));
      if (!ok) break;
      --flying;
      const uint32_t lost = bad & 3u;
      bad >>= 2;
      const uint32_t rec = ring + stage * C::kStage;
      // halves of a pair of statistics that belong to cached tokens: of keys key + 16 i, + 8
      auto kept = [&](int i) {
        const int at = key + kKv4Tile * i, len = lost >> i & 1u ? 0 : seg.s.len;
        return (at < len ? 0x0000ffffu : 0u) | (at + 8 < len ? 0xffff0000u : 0u);
      };
      // one record after the other, or with HALF both at once
#pragma unroll kUnroll
      for (int r = 0; r < (HALF ? 1 : kPair); ++r) {
        const uint32_t base = rec + r * C::kRecord;
        const int mine_of = HALF ? t4 >> 1 : r;  // the record of the lane's columns
        const uint32_t own = HALF ? rec + mine_of * C::kRecord : base;
        const int last = key - g8 + kKv4Tile * (HALF ? kPair : r + 1) - 1;
        const bool edge = last > all_see || lost != 0;

        // ---- scores
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[nt][e] = 0.0f;
        // the minima of key g8 (+ 8) and group t4: once for each piece of the sums (three, and a zero)
#pragma unroll
        for (int i = 0; i < Q; ++i)
#pragma unroll
          for (int m = 0; m < MINS; ++m) {
            uint32_t kl = G % 4 == 0 || 4 * m + t4 < G
                              ? lds_word(base + i * C::kRecord + 17 * D + (g8 * G + 4 * m + t4) * 4) : 0u;
            if (HALF && edge) kl &= kept(i);  // a NaN would reach the other record's columns
            const uint32_t a0 = __byte_perm(kl, kl, 0x1010), a1 = __byte_perm(kl, kl, 0x3232);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t q0, q1;
              lds_pair(q0, q1, qms + ((i * NT + nt) * MINS + m) * 256);
              mma_bf16_full(x[nt], a0, a1, a0, a1, q0, q1);
            }
          }
        uint32_t ks[G], vs[G], vm[Q][2];
        lds_words<G>(ks, own + 16 * D + g8 * G * 4);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          const float s0 = lo16(ks[gr]), s1 = hi16(ks[gr]);
          float acc[NT][4];
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            uint32_t w0, w1;
            lds_pair(w0, w1, base + i * C::kRecord + gr * 256 + lane * 8);
            const Codes c0 = codes_of(w0), c1 = codes_of(w1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t q[4];
              lds_words<4>(q, qs + ((i * NT + nt) * G + gr) * 512);
              if (i == 0) mma_f16_first(acc[nt], c0.n[0], c1.n[0], c0.n[1], c1.n[1], q[0], q[1]);
              else mma_f16(acc[nt], c0.n[0], c1.n[0], c0.n[1], c1.n[1], q[0], q[1]);
              mma_f16(acc[nt], c0.n[2], c1.n[2], c0.n[3], c1.n[3], q[2], q[3]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            x[nt][0] = fmaf(s0, acc[nt][0], x[nt][0]);
            x[nt][1] = fmaf(s0, acc[nt][1], x[nt][1]);
            x[nt][2] = fmaf(s1, acc[nt][2], x[nt][2]);
            x[nt][3] = fmaf(s1, acc[nt][3], x[nt][3]);
          }
        }
        lds_words<G>(vs, own + 18 * D + g8 * G * 4);
        // (lanes behind group G read the last one's again: rows that nothing uses)
#pragma unroll
        for (int i = 0; i < Q; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            vm[i][e] = lds_word(base + i * C::kRecord + 19 * D + min(g8, G - 1) * 32 + 16 * e + t4 * 4);
        bool hidden = false;  // NaN scales beside keys that some row does not see
        if (edge) {
          // keys behind the cached ones hold anything: no scale or minimum of
          // theirs counts; keys that a row does not see get -inf
          const int at = key + kKv4Tile * mine_of;
          const uint32_t keep = kept(mine_of);
          uint32_t top = 0;
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            vs[gr] &= keep;
            top = __vmaxu2(top, vs[gr]);
          }
          hidden = __any_sync(kFull, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at + (e & 2) * 4 > limit[nt][e & 1] || !(keep >> (e & 2) * 8 & 1u)) x[nt][e] = -INFINITY;
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            const int which = HALF ? i : r;
            const int pair = key - g8 + kKv4Tile * which + 2 * t4, len = lost >> which & 1u ? 0 : seg.s.len;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              vm[i][e] &= (pair + 8 * e < len ? 0x0000ffffu : 0u) | (pair + 8 * e + 1 < len ? 0xffff0000u : 0u);
          }
        }
        // ---- weights; a new reference where p * s would pass 2^15. The bound of s
        // is each key's own, over its groups
        float pr[NT][4];
        bool over = false;
        uint32_t top = kMinScale | kMinScale << 16;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) top = __vmaxu2(top, vs[gr]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[nt][e] = ex2_approx(fmaf(x[nt][e], fac[nt][e & 1], -ref[nt][e & 1]));
          const float m0 = fmaxf(pr[nt][0], pr[nt][1]) * lo16(top), m1 = fmaxf(pr[nt][2], pr[nt][3]) * hi16(top);
          over |= !(m0 < kRoom) || !(m1 < kRoom);  // NaN scales too
        }
        if (__any_sync(kFull, over)) {
          uint32_t t0 = kMinScale, t1 = kMinScale;  // NaN scales left out
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const uint32_t a = vs[gr] & 0xffffu, b = vs[gr] >> 16;
            t0 = max(t0, a < 0x7f80u ? a : 0u);
            t1 = max(t1, b < 0x7f80u ? b : 0u);
          }
          const float b0 = (float)((int)(t0 >> 7) - 126), b1 = (float)((int)(t1 >> 7) - 126);  // log2 of the keys' scales
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float m = fmaxf(kNone, fmaxf(fmaf(x[nt][j], fac[nt][j], b0), fmaf(x[nt][2 + j], fac[nt][j], b1)));
              if (HALF) m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));  // one reference for a row's two columns
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
              const float next = fmaxf(ref[nt][j], m - kHead);
              const float f = ex2_approx(ref[nt][j] - next);
              ref[nt][j] = next;
              sum[nt][j] *= f;
#pragma unroll
              for (int q = 0; q < 2 * G; ++q) {
                o[nt][q][j] *= f;
                o[nt][q][2 + j] *= f;
              }
              omin[nt][j] *= f;
              if (HALF) omin[nt][2 + j] *= f;
              pr[nt][j] = ex2_approx(fmaf(x[nt][j], fac[nt][j], -next));
              pr[nt][2 + j] = ex2_approx(fmaf(x[nt][2 + j], fac[nt][j], -next));
            }
        }
        // ---- O^T += V^T P^T
        // with HALF record 1's weights move to the rows' own columns; what record 0's
        // and they leave in columns 4 .. 7 is never read
        auto of = [&](uint32_t v, int i) { return i ? __shfl_xor_sync(kFull, v, 16) : v; };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float(&pe)[4] = pr[nt];
          sum[nt][0] += pe[0] + pe[2];
          sum[nt][1] += pe[1] + pe[3];
          // the minimum's weights in two bf16 steps (16 bits): the minimum and
          // the codes' part cancel, so a single one would show in the result
          uint32_t h0 = __byte_perm(__float_as_uint(pe[0]), __float_as_uint(pe[1]), 0x7632);
          uint32_t h1 = __byte_perm(__float_as_uint(pe[2]), __float_as_uint(pe[3]), 0x7632);
          const uint32_t l0 = transpose8(pack_bf16x2(pe[0] - lo16(h0), pe[1] - hi16(h0)));
          const uint32_t l1 = transpose8(pack_bf16x2(pe[2] - lo16(h1), pe[3] - hi16(h1)));
          h0 = transpose8(h0);
          h1 = transpose8(h1);
          if (HALF) {  // rows 0 .. 7: record 0's minima, right in columns 0 .. 3; 8 .. 15: record 1's, in 4 .. 7
            mma_bf16_full(omin[nt], vm[0][0], vm[Q - 1][0], vm[0][1], vm[Q - 1][1], h0, h1);
            mma_bf16_full(omin[nt], vm[0][0], vm[Q - 1][0], vm[0][1], vm[Q - 1][1], l0, l1);
          } else {
            mma_bf16(omin[nt], vm[0][0], vm[0][1], h0, h1);
            mma_bf16(omin[nt], vm[0][0], vm[0][1], l0, l1);
          }
        }
        auto values = [&](auto masked) {
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const float s0 = lo16(vs[gr]), s1 = hi16(vs[gr]);
            Codes c0[Q], c1[Q];
#pragma unroll
            for (int i = 0; i < Q; ++i) {
              uint32_t a, b;
              lds_pair(a, b, base + i * C::kRecord + 8 * D + gr * 256 + lane * 8);
              c0[i] = codes_of(a);
              c1[i] = codes_of(b);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float(&pe)[4] = pr[nt];
              float w[4] = {pe[0] * s0, pe[1] * s0, pe[2] * s1, pe[3] * s1};
              if (decltype(masked)::value) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (x[nt][e] == -INFINITY) w[e] = 0.0f;
              }
              const uint32_t p0 = transpose8(pack_f16x2(w[0], w[1])), p1 = transpose8(pack_f16x2(w[2], w[3]));
#pragma unroll
              for (int i = 0; i < Q; ++i) {
                const uint32_t q0 = of(p0, i), q1 = of(p1, i);
                mma_f16(o[nt][2 * gr], c0[i].n[0], c0[i].n[1], c1[i].n[0], c1[i].n[1], q0, q1);
                mma_f16(o[nt][2 * gr + 1], c0[i].n[2], c0[i].n[3], c1[i].n[2], c1[i].n[3], q0, q1);
              }
            }
          }
        };
        // a NaN group reaches only the rows that see its key
        if (!hidden) values(std::false_type());
        else values(std::true_type());
      }
      // ---- the stage is free
      __syncwarp();
      issue();
      phase ^= (uint32_t)stage;
      stage ^= 1;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (atomicCAS(p.status, 0, ATTN_ERR_TIMEOUT) == 0) p.status[1] = 0x501;
    }

    // ---- join the warps
    if (HALF) {  // first a row's two columns: their reference is one
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sum[0][j] += __shfl_xor_sync(kFull, sum[0][j], 2);
        omin[0][j] += __shfl_xor_sync(kFull, omin[0][2 + j], 2);
      }
    }
    const bool column = !HALF || t4 < 2;  // the lane's columns are rows
    float2* const my_rl = rl + turn * W * COLS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[nt][j] += __shfl_xor_sync(kFull, sum[nt][j], d);
        if (g8 == 0 && column) my_rl[warp * COLS + nt * 8 + 2 * t4 + j] = make_float2(ref[nt][j], sum[nt][j]);
      }
    __syncthreads();
    // O of the upper half of the warps, then the lower half's added to it
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      if (warp / (W / 2) == half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = (nt * 8 + 2 * t4 + j) % COLS;
            float top = my_rl[col].x;
#pragma unroll
            for (int w = 1; w < W; ++w) top = fmaxf(top, my_rl[w * COLS + col].x);
            const float f = ex2_approx(ref[nt][j] - top);
            const float f0 = f * 16777216.0f, f1 = f * 1048576.0f;  // 2^24, and a sixteenth of it
            float* const to = join + (warp % (W / 2) * COLS + col) * D + 4 * g8;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
              const float lo = f * __shfl_sync(kFull, omin[nt][j], gr * 4 + t4);
              float4 v = make_float4(fmaf(f0, o[nt][2 * gr][j], lo), fmaf(f1, o[nt][2 * gr][2 + j], lo),
                                     fmaf(f0, o[nt][2 * gr + 1][j], lo), fmaf(f1, o[nt][2 * gr + 1][2 + j], lo));
              float4* const at = reinterpret_cast<float4*>(to + 32 * gr);
              if (half == 0 && column) {
                const float4 u = *at;
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
              }
              if (column) *at = v;
            }
          }
      }
      __syncthreads();
    }
    const bool whole = seg.t0 == 0 && seg.t1 == seg.s.pairs;
    const size_t slot = 2 * (size_t)blockIdx.x + (seg.t0 > 0 ? 0 : 1);
    for (int i = threadIdx.x; i < COLS * (D / 4); i += W * 32) {
      const int col = i / (D / 4), c4 = i % (D / 4);
      const int r = seg.rb * COLS + col;
      float top = my_rl[col].x, l = 0.0f;
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, my_rl[w * COLS + col].x);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W / 2; ++w) {
        const float4 v = reinterpret_cast<const float4*>(join + (w * COLS + col) * D)[c4];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
#pragma unroll
      for (int w = 0; w < W; ++w) l += my_rl[w * COLS + col].y * ex2_approx(my_rl[w * COLS + col].x - top);
      if (!whole) {
        reinterpret_cast<float4*>(p.part_o + (slot * COLS + col) * D)[c4] = a;
        if (c4 == 0) p.part_rl[slot * COLS + col] = make_float2(top, l);
      } else if (r < seg.s.n * p.group) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int tok = seg.s.first + r / p.group, head = seg.h * p.group + r % p.group;
        reinterpret_cast<uint2*>(p.o + ((size_t)tok * p.Hq + head) * D)[c4] =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (c4 == 0)
          p.lse[(size_t)head * p.c.total + tok] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
      }
    }
    if (left <= 0 || !next_segment<COLS>(p, seg)) break;
    left = end_segment(p, seg, left);
    turn ^= 1;
  }
  if (!ok) {  // its own copies in flight still land in this shared memory
    volatile int no_abort = 0;
    for (; flying > 0; --flying) {
      bounded_wait(bars + 8 * stage, phase, &no_abort, p.timeout_ns);
      phase ^= (uint32_t)stage;
      stage ^= 1;
    }
  }
}

// Joins the partial results of the row block that border `blockIdx.x + 1` cuts
// first: O = sum_c 2^(R_c - R) O_c / sum_c 2^(R_c - R) l_c. A thread has four
// channels of a column (query row) and a slice of the parts.
constexpr int kMergeThreads = 1024;
template <int D, int COLS>
__global__ void __launch_bounds__(kMergeThreads) attn_kv4_merge_kernel(const __grid_constant__ Kv4Params p) {
  constexpr int T = D / 4, COLUMN = COLS * T, SLICES = kMergeThreads / COLUMN;
  __shared__ float4 acc[SLICES][COLUMN];
  __shared__ float tops[SLICES][COLS], sums[SLICES][COLS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 a = p.split[2 * (blockIdx.x + 1)], z = p.split[2 * (blockIdx.x + 1) + 1];
  if (a.x == 0) return;
  const int slice = threadIdx.x / COLUMN, at = threadIdx.x % COLUMN, col = at / T, c4 = at % T;
  const int r = z.x * COLS + col;
  const bool live = slice < SLICES && r < z.z * p.group;
  // parts: the last slot of CTA a.y, then the first slots of a.y + 1 .. a.z
  float top = kNone, l = 0.0f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
#pragma unroll 4
    for (int c = a.y + slice; c <= a.z; c += SLICES) {
      const size_t part = (size_t)(2 * c + (c == a.y ? 1 : 0)) * COLS + col;
      const float2 rl = p.part_rl[part];
      const float4 x = reinterpret_cast<const float4*>(p.part_o + part * D)[c4];
      const float next = fmaxf(top, rl.x), f = ex2_approx(top - next), g = ex2_approx(rl.x - next);
      top = next;
      l = l * f + rl.y * g;
      v = make_float4(v.x * f + x.x * g, v.y * f + x.y * g, v.z * f + x.z * g, v.w * f + x.w * g);
    }
    acc[slice][at] = v;
    if (c4 == 0) {
      tops[slice][col] = top;
      sums[slice][col] = l;
    }
  }
  __syncthreads();
  if (slice != 0 || !live) return;
#pragma unroll
  for (int i = 1; i < SLICES; ++i) top = fmaxf(top, tops[i][col]);
  l = 0.0f;
  v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < SLICES; ++i) {
    const float f = ex2_approx(tops[i][col] - top);
    const float4 x = acc[i][at];
    l += f * sums[i][col];
    v = make_float4(v.x + f * x.x, v.y + f * x.y, v.z + f * x.z, v.w + f * x.w);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = z.y + r / p.group, head = a.w * p.group + r % p.group;
  reinterpret_cast<uint2*>(p.o + ((size_t)tok * p.Hq + head) * D)[c4] =
      make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
  if (c4 == 0) p.lse[(size_t)head * p.c.total + tok] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

// Most column tiles of 8 rows in one pass over a kv head's records: as many as
// their accumulators leave registers for.
constexpr int max_tiles(int d) { return d <= 128 ? 2 : 1; }

// Columns for a sequence's rows: 4, or the tiles that share them evenly among
// the fewest passes.
int row_cols(int d, long long rows) {
  if (rows <= 4) return 4;
  const long long tiles = (rows + 7) / 8, passes = (tiles + max_tiles(d) - 1) / max_tiles(d);
  return 8 * (int)((tiles + passes - 1) / passes);
}

// Most CTAs of a launch: those that are resident at once.
int max_ctas(int d, int cols) { return 148 * kv4_ctas(d, cols); }

struct Kv4Workspace {
  size_t rl, split, total;
};
Kv4Workspace workspace(int d, int cols) {
  const size_t slots = 2 * (size_t)max_ctas(d, cols) * cols;
  Kv4Workspace w;
  w.rl = slots * d * 4;
  w.split = w.rl + slots * sizeof(float2);
  w.total = (w.split + 2 * (size_t)max_ctas(d, cols) * sizeof(int4) + 255) / 256 * 256;
  return w;
}

template <int D, int COLS>
cudaError_t launch_kv4(const Kv4Params& p, int ctas, cudaStream_t stream) {
  using C = Kv4Cfg<D, COLS>;
  cudaError_t e = max_dynamic_smem_once<attn_kv4_kernel<D, COLS>>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  attn_kv4_kernel<D, COLS><<<ctas, C::kWarps * 32, C::kSmemBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1 || p.whole) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas - 1);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_kv4_merge_kernel<D, COLS>, p);
}

template <int D>
cudaError_t launch_cols(const Kv4Params& p, int cols, int ctas, cudaStream_t stream) {
  if (cols == 4) return launch_kv4<D, 4>(p, ctas, stream);
  if constexpr (max_tiles(D) >= 2) {
    if (cols == 16) return launch_kv4<D, 16>(p, ctas, stream);
  }
  return launch_kv4<D, 8>(p, ctas, stream);
}

}  // namespace
}  // namespace attn_sm100

using namespace attn_sm100;

extern "C" {

size_t attn_fwd_kv4_workspace_size(int Hq, int Hkv, int max_seqlen_q, int d) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || max_seqlen_q <= 0 || (d != 64 && d != 96 && d != 128 && d != 256)) return 0;
  return workspace(d, row_cols(d, (long long)max_seqlen_q * (Hq / Hkv))).total;
}

attn_status_t attn_fwd_kv4(const void* q, const void* pool, const int* page_table, const int* seq_lens,
                           const int* cu_seqlens_q, void* o, float* lse, int num_seqs, int max_pages, int num_pages,
                           int page_size, int max_seqlen_q, int total_q, int Hq, int Hkv, int d, int causal,
                           float scale, void* workspace_ptr, size_t workspace_bytes, void* stream) {
  if (!q || !o || !lse || Hq <= 0 || Hkv <= 0 || Hq % Hkv || max_seqlen_q <= 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!isfinite(scale) || !(scale > 0.0f)) return ATTN_ERR_INVALID_ARG;
  Kv4Params p;
  const attn_status_t s = kv4_pool_params(&p.c, pool, page_table, seq_lens, cu_seqlens_q, num_seqs, max_pages,
                                          num_pages, page_size, total_q, Hkv, d);
  if (s != ATTN_OK) return s;
  if (Hq > 65535) return ATTN_ERR_UNSUPPORTED;
  if ((long long)total_q * (Hq / Hkv) > 0x7fffff00LL) return ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(lse)) & 15u)
    return ATTN_ERR_ALIGNMENT;
  const int cols = row_cols(d, (long long)max_seqlen_q * (Hq / Hkv));
  p.group = Hq / Hkv;
  // Short caches are not split: a merge and its launch take longer than the
  // pairs, or than their last ones where the row blocks fill the GPU. One query
  // row of 32 / 8 heads, whole / split (us): 500 tokens, 1 sequence 10.4 / 10.4,
  // 4 10.4 / 14.6, 64 20.6 / 24.7, 250 50 / 61; 1000 tokens, 1 14.5 / 11.0,
  // 4 14.5 / 15.0, 64 28.8 / 30.8, 250 74 / 82; 2000 tokens, 64 46 / 43, 250 119 / 115
  const long long pairs = std::max(1LL, ((long long)max_pages * page_size + kPair * kKv4Tile - 1) / (kPair * kKv4Tile));
  const long long row_blocks = std::max<long long>(num_seqs, (long long)total_q * p.group / cols) * Hkv;
  p.whole = pairs <= kAlwaysWhole || (pairs <= 32 && row_blocks >= 2 * 148);
  const Kv4Workspace w = workspace(d, cols);
  // the partial results' only; caches of kAlwaysWhole pairs never leave any
  const bool unused = pairs <= kAlwaysWhole && !workspace_ptr;
  if (!unused &&
      (!workspace_ptr || (reinterpret_cast<uintptr_t>(workspace_ptr) & 15u) || workspace_bytes < w.total))
    return ATTN_ERR_WORKSPACE;
  p.status = device_status_word();
  if (!p.status) return ATTN_ERR_CUDA;
  uint8_t* const ws = static_cast<uint8_t*>(workspace_ptr);
  p.q = static_cast<const uint16_t*>(q);
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_rl = reinterpret_cast<float2*>(ws + w.rl);
  p.split = reinterpret_cast<int4*>(ws + w.split);
  p.Hq = Hq;
  p.causal = causal;
  p.min_units = p.whole ? 1 : 8;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.timeout_ns = wait_budget_ns();
  // no more CTAs than the longest possible caches have ranges
  const long long most = ((long long)total_q * p.group / cols + num_seqs) * Hkv * (p.whole ? 1 : pairs);
  const int ctas = (int)std::max(1LL, std::min<long long>(max_ctas(d, cols), most / p.min_units));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (d) {
    case 64: e = launch_cols<64>(p, cols, ctas, st); break;
    case 96: e = launch_cols<96>(p, cols, ctas, st); break;
    case 128: e = launch_cols<128>(p, cols, ctas, st); break;
    default: e = launch_cols<256>(p, cols, ctas, st); break;
  }
  return cuda_error_status(e);
}

}  // extern "C"
