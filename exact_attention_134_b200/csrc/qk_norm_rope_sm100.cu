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
// row as 16-byte chunks, two a lane, chosen so that both values of every
// rotated pair are in one lane; the mean is a shuffle within the group. A
// group keeps its token and walks over the heads, so an angle is computed once
// for all of them: in 64 bits (position * frequency / 2 pi, reduced to a
// fraction of a turn), since in 32 bits a position of 2^17 leaves an angle
// with an error of 2^-7.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "attn_internal.h"
#include "sm100_ptx.cuh"

namespace attn_sm100 {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxAxes = 4;

struct RopeParams {
  const uint16_t* x[2];    // q, k: bf16 rows (batch, head, token strides below)
  const uint16_t* dy[2];   // gradients of the results (backward)
  uint16_t* y[2];          // results; backward: gradients of x
  const void* w[2];        // norm weights [d], or null: no norm
  const int* pos;          // positions [axes][B][N] with the strides below
  const float* inv_freq;   // [rot / 2]
  float* dw_part;          // backward: [gridDim.x * gridDim.y][2][d] sums of a block's rows
  long long xs[2][3], dys[2][3], ys[2][3];  // batch, head, token strides (elements)
  long long pos_axis, pos_batch;
  int H[2];
  int B, N, rot, heads_per_split;
  int w_bf16;
  float eps;
  int first_pair[kMaxAxes];  // pairs from first_pair[a] on turn with axis a
  int axes;
};

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r[i] << 16);
    f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Lanes of a row's group.
template <int D>
constexpr int row_lanes() {
  return D <= 64 ? 4 : D <= 128 ? 8 : 16;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rotates the lane's 16 values: pairs (i, 8 + i), or side by side.
template <bool INTER>
__device__ __forceinline__ void rotate(float* v, const float* cs, const float* sn, float sign) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : 8 + i;
    const float a = v[ia], b = v[ib], s = sign * sn[i];
    v[ia] = a * cs[i] - b * s;
    v[ib] = a * s + b * cs[i];
  }
}

template <int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int L = row_lanes<D>();
  constexpr int kRows = kThreads / L;      // tokens of a block at a time
  constexpr int U = BWD ? 2 : 4;           // rows a lane has in flight
  const int lane = threadIdx.x % L, sub = threadIdx.x / L;
  const bool holds = lane < D / 16;        // d = 96: 6 lanes of 8
  const int half = p.rot / 2;
  // the lane's two chunks of 8 values
  const bool turns = holds && lane < p.rot / 16;
  const int c0 = turns ? lane : p.rot / 8 + 2 * (lane - p.rot / 16);
  const int c1 = turns ? lane + p.rot / 16 : c0 + 1;

  float dw[2][16];
  if (BWD) {
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[0][i] = dw[1][i] = 0.0f;
  }
  const int heads = p.H[0] + p.H[1];
  const int h_begin = blockIdx.y * p.heads_per_split;
  const int h_end = min(heads, h_begin + p.heads_per_split);
  const long long rows = (long long)p.B * p.N;

  for (long long row0 = (long long)blockIdx.x * kRows; row0 < rows; row0 += (long long)gridDim.x * kRows) {
    const bool live = row0 + sub < rows;
    const long long row = live ? row0 + sub : rows - 1;
    const int b = (int)(row / p.N), n = (int)(row % p.N);
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.0f;
      sn[i] = 0.0f;
      if (turns) {
        const int pair = INTER ? (i < 4 ? 4 * c0 + i : 4 * c1 + i - 4) : 8 * lane + i;
        int axis = 0;
#pragma unroll
        for (int a = 1; a < kMaxAxes; ++a) axis += (a < p.axes && pair >= p.first_pair[a]) ? 1 : 0;
        const double turn = (double)__ldg(p.pos + axis * p.pos_axis + b * p.pos_batch + n) *
                            ((double)__ldg(p.inv_freq + min(pair, half - 1)) * 0.15915494309189533577);
        sincospif(2.0f * (float)(turn - rint(turn)), &sn[i], &cs[i]);
      }
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {  // queries, then keys
      const int first = part ? p.H[0] : 0;
      const int lo = max(h_begin, first), hi = min(h_end, first + p.H[part]);
      if (lo >= hi) continue;
      const bool norm = p.w[part] != nullptr;
      float w[16];
      if (norm && holds) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 8 * (i < 8 ? c0 : c1) + i % 8;
          w[i] = p.w_bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.w[part]) + c) << 16)
                          : __ldg(static_cast<const float*>(p.w[part]) + c);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 1.0f;
      }
      const uint16_t* const x = p.x[part] + b * p.xs[part][0] + n * p.xs[part][2];
      const uint16_t* const dy = BWD ? p.dy[part] + b * p.dys[part][0] + n * p.dys[part][2] : nullptr;
      uint16_t* const y = p.y[part] + b * p.ys[part][0] + n * p.ys[part][2];
      for (int h = lo - first; h < hi - first; h += U) {
        uint4 xa[U], xb[U], da[U], db[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          xa[u] = xb[u] = da[u] = db[u] = make_uint4(0, 0, 0, 0);
          if (holds && h + u < hi - first) {
            const uint16_t* const r = x + (h + u) * p.xs[part][1];
            if (!BWD || norm) {
              xa[u] = __ldcs(reinterpret_cast<const uint4*>(r + 8 * c0));
              xb[u] = __ldcs(reinterpret_cast<const uint4*>(r + 8 * c1));
            }
            if (BWD) {
              const uint16_t* const g = dy + (h + u) * p.dys[part][1];
              da[u] = __ldcs(reinterpret_cast<const uint4*>(g + 8 * c0));
              db[u] = __ldcs(reinterpret_cast<const uint4*>(g + 8 * c1));
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h + u >= hi - first) break;  // the same for the whole block
          float v[16];
          unpack8(xa[u], v);
          unpack8(xb[u], v + 8);
          float rstd = 1.0f;
          if (norm) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s = fmaf(v[i], v[i], s);
            rstd = rsqrtf(group_sum<L>(s) * (1.0f / D) + p.eps);
          }
          if (!BWD) {
            if (norm) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = v[i] * rstd * w[i];
            }
            rotate<INTER>(v, cs, sn, 1.0f);
          } else {
            float g[16];
            unpack8(da[u], g);
            unpack8(db[u], g + 8);
            rotate<INTER>(g, cs, sn, -1.0f);
            if (norm) {
              float s = 0.0f;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                v[i] *= rstd;
                if (live) dw[part][i] = fmaf(g[i], v[i], dw[part][i]);
                g[i] *= w[i];
                s = fmaf(g[i], v[i], s);
              }
              s = group_sum<L>(s) * (1.0f / D);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = rstd * fmaf(-v[i], s, g[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = g[i];
            }
          }
          if (holds && live) {
            uint16_t* const r = y + (h + u) * p.ys[part][1];
            __stcs(reinterpret_cast<uint4*>(r + 8 * c0), pack8(v));
            __stcs(reinterpret_cast<uint4*>(r + 8 * c1), pack8(v + 8));
          }
        }
      }
    }
  }
  if (BWD && p.dw_part != nullptr) {
    // the block's rows, in the order of its groups: the same sum every time
    __shared__ float part_sum[kRows][D];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      if (holds) {
#pragma unroll
        for (int i = 0; i < 16; ++i) part_sum[sub][8 * (i < 8 ? c0 : c1) + i % 8] = dw[part][i];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += part_sum[r][c];
        p.dw_part[(((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 + part) * D + c] = s;
      }
      __syncthreads();
    }
  }
}

// dw[part][c] = sum over the blocks' rows: 32 columns a block, 8 slices of the
// blocks summed on their own and then joined, in a fixed order.
constexpr int kSlices = 8;
__global__ void __launch_bounds__(32 * kSlices) qk_norm_rope_dw_kernel(const float* __restrict__ parts, int blocks, int d,
                                                                       float* dwq, float* dwk) {
  __shared__ float s[kSlices][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;  // c < 2 d: d is a multiple of 32
  float v = 0.0f;
  for (int i = slice; i < blocks; i += kSlices) v += parts[(size_t)i * 2 * d + c];
  s[slice][threadIdx.x % 32] = v;
  __syncthreads();
  if (slice == 0) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) v += s[i][threadIdx.x];
    if (c < d) dwq[c] = v;
    else dwk[c - d] = v;
  }
}

struct RopeGrid {
  int x, y, heads_per_split;
};

// Forward: a block for every group of tokens, the heads split over blocks
// while they are too few to fill the GPU. Backward: at most four blocks an SM,
// each walking over many tokens, since every block leaves a row of weight
// gradients to be added up.
RopeGrid rope_grid(int B, int N, int heads, int d, bool bwd) {
  const int rows = kThreads / (d <= 64 ? 4 : d <= 128 ? 8 : 16);
  const long long blocks = ((long long)B * N + rows - 1) / rows;
  const long long fill = 148 * 4;
  RopeGrid g;
  g.x = (int)std::min<long long>(blocks, bwd ? fill : 0x7fffffffLL);
  const int want = (int)std::min<long long>(heads, std::max<long long>(1, fill / g.x));
  g.heads_per_split = (heads + want - 1) / want;
  g.y = (heads + g.heads_per_split - 1) / g.heads_per_split;
  return g;
}

template <bool INTER, bool BWD>
void launch_rope(const RopeParams& p, const RopeGrid& g, int d, cudaStream_t stream) {
  const dim3 grid(g.x, g.y);
  switch (d) {
    case 64: qk_norm_rope_kernel<64, INTER, BWD><<<grid, kThreads, 0, stream>>>(p); break;
    case 96: qk_norm_rope_kernel<96, INTER, BWD><<<grid, kThreads, 0, stream>>>(p); break;
    case 128: qk_norm_rope_kernel<128, INTER, BWD><<<grid, kThreads, 0, stream>>>(p); break;
    default: qk_norm_rope_kernel<256, INTER, BWD><<<grid, kThreads, 0, stream>>>(p); break;
  }
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

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
  if (Hq > 65535 || Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
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
  p.x[0] = static_cast<const uint16_t*>(q);
  p.x[1] = static_cast<const uint16_t*>(k);
  p.y[0] = static_cast<uint16_t*>(q_out);
  p.y[1] = static_cast<uint16_t*>(k_out);
  copy_strides(p.xs, strides);
  copy_strides(p.ys, strides + 6);
  const RopeGrid g = rope_grid(B, N, Hq + Hkv, d, false);
  p.heads_per_split = g.heads_per_split;
  if (interleaved) launch_rope<true, false>(p, g, d, static_cast<cudaStream_t>(stream));
  else launch_rope<false, false>(p, g, d, static_cast<cudaStream_t>(stream));
  return cuda_error_status(cudaGetLastError());
}

size_t attn_qk_norm_rope_bwd_workspace_size(int B, int N, int Hq, int Hkv, int d) {
  if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || (d != 64 && d != 96 && d != 128 && d != 256)) return 0;
  const RopeGrid g = rope_grid(B, N, Hq + Hkv, d, true);
  return ((size_t)g.x * g.y * 2 * d * sizeof(float) + 255) / 256 * 256;
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
  const RopeGrid g = rope_grid(B, N, Hq + Hkv, d, true);
  p.heads_per_split = g.heads_per_split;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (interleaved) launch_rope<true, true>(p, g, d, st);
  else launch_rope<false, true>(p, g, d, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !q_weight) return cuda_error_status(e);
  qk_norm_rope_dw_kernel<<<2 * d / 32, 32 * kSlices, 0, st>>>(p.dw_part, g.x * g.y, d, dq_weight, dk_weight);
  return cuda_error_status(cudaGetLastError());
}

}  // extern "C"
