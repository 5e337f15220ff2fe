// qk_norm_rope_sm100.cu — queries and keys between their projection and
// attention: the RMS norm of every head and the rotation by the position, in
// one pass, and its gradients.
//
//   xhat = x / sqrt(mean(x^2) + eps),  n = xhat * w          (w: [d], shared by the heads)
//   pair i of n, (a, b): a' = a cos t - b sin t, b' = a sin t + b cos t,
//   t = position[axis of i] * inv_freq[i]
// and, for the gradient dy of the result y,
//   dn = the rotation of dy by -t,  dw = sum over rows of dn * xhat,
//   g = dn * w,  dx = (g - xhat * mean(g * xhat)) / sqrt(mean(x^2) + eps).
//
// HBM-bound: 4 bytes a value forwards (bf16 read, written), 6 backwards; the
// norm stays in fp32 between the two steps and is rounded once, at the end.
// A group of lanes (d / 16 of them, rounded up to a power of two) holds one
// row as two chunks of 8 values a lane, chosen so that both values of every
// rotated pair are in one lane; the mean is a shuffle within the group. A
// warp keeps its tokens and walks over their heads, so an angle is computed
// once for many of them: in 64 bits (position * frequency / 2 pi, reduced to a
// fraction of a turn), since in 32 bits a position of 2^17 leaves an angle
// with an error of 2^-7. The instructions of a row came to bound it (scalar
// arithmetic and loads straight into registers: 75 us forwards, 133 backwards
// where the bytes take 51 and 77), hence packed fp32x2 arithmetic, 16 values a
// lane against the loop's overhead, and rows copied ahead into shared memory
// by cp.async, which keeps 48 KB an SM in flight without registers.
// Measured (B200, one call behind the other): 2 x 8192 x 40 heads of 128,
// forwards 63 us (5.3 TB/s), backwards 88 us (5.7 TB/s, both launches).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "attn_internal.h"
#include "sm100_rows.cuh"

namespace attn_sm100 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;
// Most tokens: their number, rounded up to a block's, is computed in 32 bits.
constexpr int kMaxTokens = 0x7fff0000;
// Blocks of an SM and steps in a warp's ring. Large blocks and little in flight
// keep a block's rows together in DRAM; more of either is slower once every
// call's results are written back behind the next one's reads. Measured, one
// call behind the other (us), threads x blocks, ring: forwards 2 x 8192 x 40
// heads of 128: 128 x 6, 4 69.9; 256 x 3, 4 69.9; 256 x 3, 2 66.0; 256 x 2, 2
// 63.6; 256 x 2, 3 62.9; 256 x 2, 4 66.0; 512 x 1, 2 64.7; backwards: 128 x 4, 3
// 98.6; 256 x 2, 3 96.2; 256 x 2, 2 87.7; 256 x 2, 1 98.5; 384 x 1, 2 89.2.
constexpr int kFwdBlocksPerSm = 2, kFwdRing = 3;
constexpr int kBwdBlocksPerSm = 2, kBwdRing = 2;

struct RopeParams {
  const uint16_t* x[2];    // q, k: bf16 rows (batch, head, token strides below)
  const uint16_t* dy[2];   // gradients of the results (backward)
  uint16_t* y[2];          // results; backward: gradients of x
  const void* w[2];        // norm weights [d], or null: no norm
  const int* pos;          // positions [axes][B][N] with the strides below
  const float* inv_freq;   // [rot / 2]
  float* dw_part;          // backward: [gridDim.x][d] sums of a block's rows
  long long xs[2][3], dys[2][3], ys[2][3];  // batch, head, token strides (elements)
  long long pos_axis, pos_batch;
  int H[2];
  int B, N, rot;
  int q_blocks;            // blocks of the queries
  int w_bf16;
  float eps;
  int first_pair[kMaxAxes];  // pairs from first_pair[a] on turn with axis a
  int axes;
};

// A lane holds 16 values of a row as 8 pairs (a, b), in packed registers of two
// neighbouring pairs each (fp32x2 arithmetic: half the instructions): the
// values of chunk 0 and of chunk 1, or those that stand side by side.
struct Pairs {
  float2 a[4], b[4];
};

template <bool INTER>
__device__ __forceinline__ void unpack(const uint4& u0, const uint4& u1, Pairs& v) {
  const uint32_t r[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s = INTER ? r[2 * i] : r[i], t = INTER ? r[2 * i + 1] : r[4 + i];
    const float sl = __uint_as_float(s << 16), sh = __uint_as_float(s & 0xffff0000u);
    const float tl = __uint_as_float(t << 16), th = __uint_as_float(t & 0xffff0000u);
    v.a[i] = INTER ? make_float2(sl, tl) : make_float2(sl, sh);
    v.b[i] = INTER ? make_float2(sh, th) : make_float2(tl, th);
  }
}

template <bool INTER>
__device__ __forceinline__ void pack(const Pairs& v, uint4& u0, uint4& u1) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {
      r[2 * i] = pack_bf16x2(v.a[i].x, v.b[i].x);
      r[2 * i + 1] = pack_bf16x2(v.a[i].y, v.b[i].y);
    } else {
      r[i] = pack_bf16x2(v.a[i].x, v.a[i].y);
      r[4 + i] = pack_bf16x2(v.b[i].x, v.b[i].y);
    }
  }
  u0 = make_uint4(r[0], r[1], r[2], r[3]);
  u1 = make_uint4(r[4], r[5], r[6], r[7]);
}

// Lanes of a row's group.
template <int D>
constexpr int row_lanes() {
  return D <= 64 ? 4 : D <= 128 ? 8 : 16;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float2 a) {
  float v = a.x + a.y;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }

// cos and sin of the lane's 8 pairs for one token.
template <bool INTER>
__device__ __forceinline__ void angles(const RopeParams& p, int c0, int c1, int b, int n, float2* cs, float2* sn) {
  const int* const pos = p.pos + b * p.pos_batch + n;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pair = INTER ? (i < 4 ? 4 * c0 + i : 4 * c1 + i - 4) : 8 * c0 + i;
    int axis = 0;
#pragma unroll
    for (int a = 1; a < kMaxAxes; ++a) axis += (a < p.axes && pair >= p.first_pair[a]) ? 1 : 0;
    const double turn = (double)__ldg(pos + axis * p.pos_axis) *
                        ((double)__ldg(p.inv_freq + pair) * 0.15915494309189533577);
    float s, c;
    sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
    if (i % 2) {
      cs[i / 2].y = c;
      sn[i / 2].y = s;
    } else {
      cs[i / 2].x = c;
      sn[i / 2].x = s;
    }
  }
}

// A step is one head of kRows tokens; the steps of the queries are shared by
// blocks 0 .. q_blocks - 1, the keys' by the others, each a range of steps
// with the heads of a group of tokens side by side. Every warp copies its own
// rows ahead into a ring in shared memory (no barrier between warps).
template <int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? kBwdBlocksPerSm : kFwdBlocksPerSm)
    qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int L = row_lanes<D>();
  constexpr int kRows = kThreads / L;      // tokens of a block at a time
  constexpr int K = BWD ? kBwdRing : kFwdRing;  // steps in the ring
  constexpr int kStep = 32 * 32 * (BWD ? 2 : 1);  // bytes of a step and warp: x, then dy
  __shared__ __align__(16) uint8_t ring[kThreads / 32 * K * kStep];
  const int lane = threadIdx.x % L, sub = threadIdx.x / L;
  const bool holds = lane < D / 16;        // d = 96: 6 lanes of 8
  // the lane's two chunks of 8 values
  const bool turns = holds && lane < p.rot / 16;
  const int c0 = turns ? lane : p.rot / 8 + 2 * (lane - p.rot / 16);
  const int c1 = turns ? lane + p.rot / 16 : c0 + 1;
  uint8_t* const mine = ring + threadIdx.x / 32 * (K * kStep);
  const int from = threadIdx.x % 32 / L * (L * 32);
  const uint32_t to = smem_addr(mine) + from + lane * 16;

  const int part = (int)blockIdx.x >= p.q_blocks ? 1 : 0;
  const int block = part ? blockIdx.x - p.q_blocks : blockIdx.x;
  const int blocks = part ? gridDim.x - p.q_blocks : p.q_blocks;
  const int heads = p.H[part], rows = p.B * p.N;
  const long long steps = (long long)((rows + kRows - 1) / kRows) * heads;
  const long long begin = steps * block / blocks;
  int left = (int)(steps * (block + 1) / blocks - begin), ahead = left;

  const bool norm = p.w[part] != nullptr;
  auto channel = [&](int i, bool b) {  // of the lane's pair i
    return INTER ? 8 * (i < 4 ? c0 : c1) + 2 * (i % 4) + b : 8 * (b ? c1 : c0) + i;
  };
  auto weight = [&](int i, bool b) {
    const int c = channel(i, b);
    return !norm || !holds ? 1.0f
           : p.w_bf16      ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.w[part]) + c) << 16)
                           : __ldg(static_cast<const float*>(p.w[part]) + c);
  };
  auto token = [&](int group, int& b, int& n) {  // false behind the last one (which stands in)
    const int row = min(group * kRows + sub, rows - 1);
    b = row / p.N;
    n = row - b * p.N;
    return group * kRows + sub < rows;
  };

  const long long hx = p.xs[part][1], hdy = BWD ? p.dys[part][1] : 0, hy = p.ys[part][1];
  int group = (int)(begin / heads), h = (int)(begin % heads), b, n;
  int next_group = group, next_h = h, stage = 0, next_stage = 0;
  bool copies = token(group, b, n) && holds;  // rows behind the last are not read: another warp may write in place
  const uint16_t* x = p.x[part] + b * p.xs[part][0] + n * p.xs[part][2] + h * hx + 8 * lane;
  const uint16_t* dy = BWD ? p.dy[part] + b * p.dys[part][0] + n * p.dys[part][2] + h * hdy + 8 * lane : nullptr;
  auto fetch = [&]() {
    if (ahead > 0) {
      --ahead;
      if (copies) {
        const uint32_t at = to + next_stage * kStep;
        if (!BWD || norm) {
          cp_async16(at, x);
          cp_async16(at + D, x + D / 2);
        }
        if (BWD) {
          cp_async16(at + 1024, dy);
          cp_async16(at + 1024 + D, dy + D / 2);
        }
      }
      x += hx;
      dy += hdy;
      if (++next_h == heads) {
        next_h = 0;
        int b_, n_;
        copies = token(++next_group, b_, n_) && holds;
        x = p.x[part] + b_ * p.xs[part][0] + n_ * p.xs[part][2] + 8 * lane;
        if (BWD) dy = p.dy[part] + b_ * p.dys[part][0] + n_ * p.dys[part][2] + 8 * lane;
      }
      if (++next_stage == K) next_stage = 0;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < K; ++i) fetch();

  Pairs w, dw;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w.a[i] = make_float2(weight(2 * i, false), weight(2 * i + 1, false));
    w.b[i] = make_float2(weight(2 * i, true), weight(2 * i + 1, true));
    dw.a[i] = dw.b[i] = both(0.0f);
  }
  float2 cs[4] = {both(1.0f), both(1.0f), both(1.0f), both(1.0f)};
  float2 sn[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
  bool fresh = true, live = false;
  uint16_t* y = nullptr;
  // the lane's chunk 1 behind chunk 0, in elements
  const int over = 8 * (c1 - c0);
  for (; left > 0; --left) {
    if (fresh) {  // another group of tokens
      live = token(group, b, n);
      y = p.y[part] + b * p.ys[part][0] + n * p.ys[part][2] + h * hy + 8 * c0;
      if (turns) angles<INTER>(p, c0, c1, b, n, cs, sn);
      fresh = false;
    }
    cp_async_wait<K - 1>();
    __syncwarp();
    const uint8_t* const s_x = mine + stage * kStep + from;
    Pairs v, g;
    unpack<INTER>(*reinterpret_cast<const uint4*>(s_x + 16 * c0), *reinterpret_cast<const uint4*>(s_x + 16 * c1), v);
    if (BWD)
      unpack<INTER>(*reinterpret_cast<const uint4*>(s_x + 1024 + 16 * c0),
                    *reinterpret_cast<const uint4*>(s_x + 1024 + 16 * c1), g);
    if (!holds || !live) {  // nothing was copied there
#pragma unroll
      for (int i = 0; i < 4; ++i) v.a[i] = v.b[i] = g.a[i] = g.b[i] = both(0.0f);
    }
    __syncwarp();
    fetch();
    if (++stage == K) stage = 0;
    float rstd = 1.0f;
    if (norm) {
      float2 s = mul2(v.a[0], v.a[0]), t = mul2(v.b[0], v.b[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        s = fma2(v.a[i], v.a[i], s);
        t = fma2(v.b[i], v.b[i], t);
      }
      rstd = rsqrtf(group_sum<L>(add2(s, t)) * (1.0f / D) + p.eps);
    }
    const float2 r = both(rstd);
    if (!BWD) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 na = mul2(v.a[i], mul2(w.a[i], r)), nb = mul2(v.b[i], mul2(w.b[i], r));
        v.a[i] = fma2(nb, neg2(sn[i]), mul2(na, cs[i]));
        v.b[i] = fma2(na, sn[i], mul2(nb, cs[i]));
      }
    } else {
      float2 s = both(0.0f), t = both(0.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 ga = g.a[i], gb = g.b[i];
        g.a[i] = fma2(gb, sn[i], mul2(ga, cs[i]));
        g.b[i] = fma2(ga, neg2(sn[i]), mul2(gb, cs[i]));
      }
      if (norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v.a[i] = mul2(v.a[i], r);
          v.b[i] = mul2(v.b[i], r);
          const float2 ta = mul2(g.a[i], v.a[i]), tb = mul2(g.b[i], v.b[i]);
          if (live) {
            dw.a[i] = add2(dw.a[i], ta);
            dw.b[i] = add2(dw.b[i], tb);
          }
          s = fma2(w.a[i], ta, s);
          t = fma2(w.b[i], tb, t);
        }
        const float2 m = both(-rstd * (group_sum<L>(add2(s, t)) * (1.0f / D)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v.a[i] = fma2(g.a[i], mul2(w.a[i], r), mul2(v.a[i], m));
          v.b[i] = fma2(g.b[i], mul2(w.b[i], r), mul2(v.b[i], m));
        }
      } else {
        v = g;
      }
    }
    if (holds && live) {
      uint4 y0, y1;
      pack<INTER>(v, y0, y1);
      __stcs(reinterpret_cast<uint4*>(y), y0);
      __stcs(reinterpret_cast<uint4*>(y + over), y1);
    }
    y += hy;
    if (++h == heads) {
      h = 0;
      ++group;
      fresh = true;
    }
  }
  if (BWD && p.dw_part != nullptr) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the block's rows, in the order of its groups: the same sum every time
    static_assert(kRows * D * 4 <= sizeof(ring), "the sums fit into the ring");
    float* const part_sum = reinterpret_cast<float*>(ring);
    __syncthreads();
    if (holds) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part_sum[sub * D + channel(2 * i, false)] = dw.a[i].x;
        part_sum[sub * D + channel(2 * i + 1, false)] = dw.a[i].y;
        part_sum[sub * D + channel(2 * i, true)] = dw.b[i].x;
        part_sum[sub * D + channel(2 * i + 1, true)] = dw.b[i].y;
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int r_ = 0; r_ < kRows; ++r_) s += part_sum[r_ * D + c];
      p.dw_part[(size_t)blockIdx.x * D + c] = s;
    }
  }
}

// dw[c] = sum over the blocks' rows: 32 columns of the queries' or the keys' a
// block, 32 slices of the blocks summed on their own and then joined, in a
// fixed order.
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices)
    qk_norm_rope_dw_kernel(const float* __restrict__ parts, int q_blocks, int blocks, int d, float* dwq, float* dwk) {
  __shared__ float s[kSlices][33];
  const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
  const bool keys = (int)blockIdx.x >= d / 32;
  const int c = blockIdx.x * 32 + lane - (keys ? d : 0);
  const int first = keys ? q_blocks : 0, last = keys ? blocks : q_blocks;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v = 0.0f;
#pragma unroll 10
  for (int i = first + slice; i < last; i += kSlices) v += parts[(size_t)i * d + c];
  s[slice][lane] = v;
  __syncthreads();
  if (slice == 0) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) v += s[i][lane];
    (keys ? dwk : dwq)[c] = v;
  }
}

struct RopeGrid {
  int blocks, q_blocks;
};

// One wave of blocks at most, shared out between queries and keys by their steps.
RopeGrid rope_grid(int B, int N, int Hq, int Hkv, int d, bool bwd) {
  const int rows = kThreads / (d <= 64 ? 4 : d <= 128 ? 8 : 16);
  const long long groups = ((long long)B * N + rows - 1) / rows, sq = groups * Hq, sk = groups * Hkv;
  const long long fill = 148LL * (bwd ? kBwdBlocksPerSm : kFwdBlocksPerSm);
  RopeGrid g;
  const long long kb = sq + sk <= fill ? sk : std::max(1LL, (fill * sk + (sq + sk) / 2) / (sq + sk));
  g.q_blocks = (int)(sq + sk <= fill ? sq : std::max(1LL, fill - kb));
  g.blocks = g.q_blocks + (int)kb;
  return g;
}

template <bool INTER, bool BWD>
void launch_rope(const RopeParams& p, const RopeGrid& g, int d, cudaStream_t stream) {
  switch (d) {
    case 64: qk_norm_rope_kernel<64, INTER, BWD><<<g.blocks, kThreads, 0, stream>>>(p); break;
    case 96: qk_norm_rope_kernel<96, INTER, BWD><<<g.blocks, kThreads, 0, stream>>>(p); break;
    case 128: qk_norm_rope_kernel<128, INTER, BWD><<<g.blocks, kThreads, 0, stream>>>(p); break;
    default: qk_norm_rope_kernel<256, INTER, BWD><<<g.blocks, kThreads, 0, stream>>>(p); break;
  }
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether the result at y may be written while x is read: another tensor, or x itself with its own strides.
bool apart(const void* x, const long long* xs, const void* y, const long long* ys) {
  return x != y || (xs[0] == ys[0] && xs[1] == ys[1] && xs[2] == ys[2]);
}

// Whether the two results are two tensors, and neither is what the other one is made of.
bool uncrossed(const void* const* x, const void* const* y) {
  return y[0] != y[1] && y[0] != x[1] && y[1] != x[0];
}

// The checks and parameters that both directions share. tensors: q, k, then
// for each further pair as the caller lists them (strides in the same order).
attn_status_t rope_params(RopeParams* p, const void* const* tensors, int num_tensors, const long long* strides,
                          const void* q_weight, const void* k_weight, int weight_bf16, const int* positions,
                          long long pos_axis_stride, long long pos_batch_stride, const float* inv_freq,
                          const int* sections, int num_axes, int rotary_dim, int interleaved, int B, int N, int Hq,
                          int Hkv, int d, float eps) {
  for (int i = 0; i < num_tensors; ++i)
    if (!tensors[i]) return ATTN_ERR_INVALID_ARG;
  if (!strides || B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0) return ATTN_ERR_INVALID_ARG;
  if ((q_weight == nullptr) != (k_weight == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (weight_bf16 != 0 && weight_bf16 != 1) return ATTN_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (q_weight && !(isfinite(eps) && eps >= 0.0f)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 96 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 16) return ATTN_ERR_INVALID_ARG;
  if (Hq > 65535 || Hkv > 65535 || (long long)B * N > kMaxTokens) return ATTN_ERR_UNSUPPORTED;
  *p = RopeParams();
  if (rotary_dim > 0) {
    if (!positions || !inv_freq || !sections || pos_axis_stride < 0 || pos_batch_stride < 0) return ATTN_ERR_INVALID_ARG;
    if (num_axes < 1 || num_axes > kMaxAxes) return ATTN_ERR_INVALID_ARG;
    int sum = 0;
    for (int a = 0; a < num_axes; ++a) {
      if (sections[a] < 0 || sections[a] > rotary_dim / 2) return ATTN_ERR_INVALID_ARG;
      p->first_pair[a] = sum;
      sum += sections[a];
    }
    if (sum != rotary_dim / 2) return ATTN_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return ATTN_ERR_ALIGNMENT;
  }
  for (int i = 0; i < num_tensors; ++i) {
    if (!aligned(tensors[i], 16)) return ATTN_ERR_ALIGNMENT;
    for (int j = 0; j < 3; ++j) {
      if (strides[3 * i + j] < 0) return ATTN_ERR_INVALID_ARG;
      if (strides[3 * i + j] % 8) return ATTN_ERR_ALIGNMENT;
    }
  }
  if (q_weight && (!aligned(q_weight, weight_bf16 ? 2 : 4) || !aligned(k_weight, weight_bf16 ? 2 : 4)))
    return ATTN_ERR_ALIGNMENT;
  p->w[0] = q_weight;
  p->w[1] = k_weight;
  p->pos = positions;
  p->inv_freq = inv_freq;
  p->pos_axis = pos_axis_stride;
  p->pos_batch = pos_batch_stride;
  p->H[0] = Hq;
  p->H[1] = Hkv;
  p->B = B;
  p->N = N;
  p->rot = rotary_dim;
  p->w_bf16 = weight_bf16;
  p->eps = eps;
  p->axes = rotary_dim > 0 ? num_axes : 0;
  return ATTN_OK;
}

void copy_strides(long long (*to)[3], const long long* from) {
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 3; ++j) to[i][j] = from[3 * i + j];
}

}  // namespace
}  // namespace attn_sm100

using namespace attn_sm100;

extern "C" {

attn_status_t attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides,
                                const void* q_weight, const void* k_weight, int weight_bf16, const int* positions,
                                long long pos_axis_stride, long long pos_batch_stride, const float* inv_freq,
                                const int* sections, int num_axes, int rotary_dim, int interleaved, int B, int N,
                                int Hq, int Hkv, int d, float eps, void* stream) {
  RopeParams p;
  const void* const t[4] = {q, k, q_out, k_out};
  const attn_status_t s =
      rope_params(&p, t, 4, strides, q_weight, k_weight, weight_bf16, positions, pos_axis_stride, pos_batch_stride,
                  inv_freq, sections, num_axes, rotary_dim, interleaved, B, N, Hq, Hkv, d, eps);
  if (s != ATTN_OK) return s;
  if (!apart(q, strides, q_out, strides + 6) || !apart(k, strides + 3, k_out, strides + 9) || !uncrossed(t, t + 2))
    return ATTN_ERR_INVALID_ARG;
  p.x[0] = static_cast<const uint16_t*>(q);
  p.x[1] = static_cast<const uint16_t*>(k);
  p.y[0] = static_cast<uint16_t*>(q_out);
  p.y[1] = static_cast<uint16_t*>(k_out);
  copy_strides(p.xs, strides);
  copy_strides(p.ys, strides + 6);
  const RopeGrid g = rope_grid(B, N, Hq, Hkv, d, false);
  p.q_blocks = g.q_blocks;
  if (interleaved) launch_rope<true, false>(p, g, d, static_cast<cudaStream_t>(stream));
  else launch_rope<false, false>(p, g, d, static_cast<cudaStream_t>(stream));
  return cuda_error_status(cudaGetLastError());
}

size_t attn_qk_norm_rope_bwd_workspace_size(int B, int N, int Hq, int Hkv, int d) {
  if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || (d != 64 && d != 96 && d != 128 && d != 256)) return 0;
  return ((size_t)rope_grid(B, N, Hq, Hkv, d, true).blocks * d * sizeof(float) + 255) / 256 * 256;
}

attn_status_t attn_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, void* dq,
                                    void* dk, const long long* strides, const void* q_weight, const void* k_weight,
                                    int weight_bf16, float* dq_weight, float* dk_weight, const int* positions,
                                    long long pos_axis_stride, long long pos_batch_stride, const float* inv_freq,
                                    const int* sections, int num_axes, int rotary_dim, int interleaved, int B, int N,
                                    int Hq, int Hkv, int d, float eps, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  RopeParams p;
  const void* const t[6] = {q, k, dq_out, dk_out, dq, dk};
  const attn_status_t s =
      rope_params(&p, t, 6, strides, q_weight, k_weight, weight_bf16, positions, pos_axis_stride, pos_batch_stride,
                  inv_freq, sections, num_axes, rotary_dim, interleaved, B, N, Hq, Hkv, d, eps);
  if (s != ATTN_OK) return s;
  if (!apart(dq_out, strides + 6, dq, strides + 12) || !apart(dk_out, strides + 9, dk, strides + 15) ||
      !uncrossed(t + 2, t + 4))
    return ATTN_ERR_INVALID_ARG;
  if (q_weight && (!apart(q, strides, dq, strides + 12) || !apart(k, strides + 3, dk, strides + 15) || !uncrossed(t, t + 4)))
    return ATTN_ERR_INVALID_ARG;
  if (q_weight) {
    if (!dq_weight || !dk_weight) return ATTN_ERR_INVALID_ARG;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return ATTN_ERR_ALIGNMENT;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d))
      return ATTN_ERR_WORKSPACE;
    p.dw_part = static_cast<float*>(workspace);
  }
  p.x[0] = static_cast<const uint16_t*>(q);
  p.x[1] = static_cast<const uint16_t*>(k);
  p.dy[0] = static_cast<const uint16_t*>(dq_out);
  p.dy[1] = static_cast<const uint16_t*>(dk_out);
  p.y[0] = static_cast<uint16_t*>(dq);
  p.y[1] = static_cast<uint16_t*>(dk);
  copy_strides(p.xs, strides);
  copy_strides(p.dys, strides + 6);
  copy_strides(p.ys, strides + 12);
  const RopeGrid g = rope_grid(B, N, Hq, Hkv, d, true);
  p.q_blocks = g.q_blocks;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (interleaved) launch_rope<true, true>(p, g, d, st);
  else launch_rope<false, true>(p, g, d, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !q_weight) return cuda_error_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * d / 32);
  cfg.blockDim = dim3(32 * kSlices);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_error_status(cudaLaunchKernelEx(&cfg, qk_norm_rope_dw_kernel, static_cast<const float*>(p.dw_part),
                                              g.q_blocks, g.blocks, d, dq_weight, dk_weight));
}

}  // extern "C"
