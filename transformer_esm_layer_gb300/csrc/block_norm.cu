// The residual stream between two blocks, in one pass over it:
//   u = dropout(post(y)),  x_out = residual_scale * x + gate * u,  h = pre(x_out)
// post: the norm after the block that made y (or none); pre: the norm before the next block (or none);
// each a LayerNorm, (z - mean) / sqrt(var + eps) * gamma + beta with the biased variance, or an RMS norm,
// z / sqrt(mean(z^2) + eps) * gamma + beta.  And its gradient.
//
// Bound by memory: 12 bytes an element forward and 18 backward with bfloat16 blocks (the residual
// stream and its gradient are float32).
#include <algorithm>

#include "dropout.cuh"
#include "internal.h"

namespace esm {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Mean and 1 / sqrt(var + eps) of a row held by W warps, G spans of 256 columns each: warp w holds spans
// w, w + W, ...  A warp's own mean and squared deviations are taken in two passes over its registers;
// those of several warps are joined with their counts (Chan, Golub, LeVeque 1979), which loses
// no digits to a large mean and takes one barrier.  slot: shared memory of this row's and norm's own.
template <bool VEC, int G>
__device__ __forceinline__ float2 row_moments(const float (&z)[G][8], const BlockNormArgs& a, int W, int w, int lane,
                                              float2* slot) {
  float s = 0.f, q = 0.f, mean = 0.f;
  int n = 0;
  if (!a.rms) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      n += min(max(a.cols - (g * W + w) * 256, 0), 256);
#pragma unroll
      for (int k = 0; k < 8; ++k) s += z[g][k];
    }
    mean = warp_sum(s) / (float)n;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int left = a.cols - (g * W + w) * 256;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = span_col<VEC>(lane, k) < left ? z[g][k] - mean : 0.f;
      q = fmaf(d, d, q);
    }
  }
  q = warp_sum(q);
  if (W > 1) {
    if (lane == 0) slot[w] = make_float2(mean, q);
    __syncthreads();
    float total = 0.f, m = 0.f;
    for (int i = 0; i < W; ++i) {
      int ni = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) ni += min(max(a.cols - (g * W + i) * 256, 0), 256);
      m = fmaf((float)ni, slot[i].x, m);
    }
    m /= (float)a.cols;
    for (int i = 0; i < W; ++i) {
      int ni = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) ni += min(max(a.cols - (g * W + i) * 256, 0), 256);
      const float d = slot[i].x - m;
      total += fmaf((float)ni * d, d, slot[i].y);
    }
    mean = m;
    q = total;
  }
  return make_float2(mean, rsqrtf(q / (float)a.cols + a.eps));
}

// W warps per row and G spans per warp; with W = 1 a block holds several rows.
template <typename T, bool VEC, int G>
__global__ void __launch_bounds__(512) block_norm_kernel(const BlockNormArgs a, int W) {
  __shared__ float2 slots[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = W > 1 ? warp : 0;
  const int row = W > 1 ? blockIdx.x : blockIdx.x * (blockDim.x >> 5) + warp;
  if (row >= a.rows) return;
  const size_t base = (size_t)row * a.cols;
  float x[G][8], u[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (g * W + w) * 256, left = a.cols - c0;
    span_load<VEC>(static_cast<const T*>(a.y) + base + c0, left, lane, u[g]);
    span_load<VEC>(a.x + base + c0, left, lane, x[g]);
  }
  const PhiloxState ps = philox_state(a.mask);
  float2 post = make_float2(0.f, 0.f), pre = make_float2(0.f, 0.f);
  if (a.post_gamma) post = row_moments<VEC, G>(u, a, W, w, lane, slots[0]);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (g * W + w) * 256, left = a.cols - c0;
    const uint32_t keep = span_keep<VEC>(a.mask, ps, (unsigned long long)row * ((a.cols + 7) / 8) + c0 / 8, lane);
    float p[8];
    if (a.post_gamma) {
      span_load<VEC>(static_cast<const T*>(a.post_gamma) + c0, left, lane, p);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[g][k] = (u[g][k] - post.x) * post.y * p[k];
      if (a.post_beta) {
        span_load<VEC>(static_cast<const T*>(a.post_beta) + c0, left, lane, p);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[g][k] += p[k];
      }
    }
    if (a.gate) span_load<VEC>(static_cast<const T*>(a.gate) + (a.gate_rows ? base : 0) + c0, left, lane, p);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v = keep >> k & 1u ? u[g][k] * a.mask.scale : 0.f;
      if (a.gate) v *= p[k];
      x[g][k] = span_col<VEC>(lane, k) < left ? fmaf(a.residual_scale, x[g][k], v) : 0.f;
    }
    span_store<VEC>(a.x_out + base + c0, left, lane, x[g]);
  }
  if (a.pre_gamma) {
    pre = row_moments<VEC, G>(x, a, W, w, lane, slots[1]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (g * W + w) * 256, left = a.cols - c0;
      float p[8];
      span_load<VEC>(static_cast<const T*>(a.pre_gamma) + c0, left, lane, p);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[g][k] = (x[g][k] - pre.x) * pre.y * p[k];
      if (a.pre_beta) {
        span_load<VEC>(static_cast<const T*>(a.pre_beta) + c0, left, lane, p);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[g][k] += p[k];
      }
      span_store<VEC>(static_cast<T*>(a.h) + base + c0, left, lane, x[g]);
    }
  }
  if (a.stats && w == 0 && lane < 4)
    a.stats[(size_t)row * 4 + lane] = lane == 0 ? post.x : lane == 1 ? post.y : lane == 2 ? pre.x : pre.y;
}

// ---- backward ----
// With xh = (x_out - mean) rstd, yh likewise, k = keep * scale * gate, g = d_h * gamma_pre:
//   G  = d_x_out + rstd_x (g - mean(g) - xh mean(g xh))        dx = residual_scale G
//   u's gradient, through gate and dropout, is k G:  dgate = keep scale G post(y),
//   dgamma_post = sum k G yh, dbeta_post = sum k G, and with c = k gamma_post
//   dy = rstd_y (c G - mean(c G) - yh mean(c G yh))
// The means over c G hold G, which holds the means over g; but G is linear in those, so with
// e = d_x_out + rstd_x g all of a row's sums
//   S1 = sum g, S2 = sum g xh, S3 = sum c e, S4 = sum c, S5 = sum c xh, S6 = sum c yh e, S7 = sum c yh,
//   S8 = sum c yh xh
// are taken in one exchange:  sum c G = S3 - rstd_x (S1 S4 + S2 S5) / cols, and so on.
//
// Eight sums over a warp: every step halves the number of values a lane still adds.  Lane l ends with
// the total of value (l / 4) with its three bits reversed by the order of the steps: l / 16 chooses the
// upper bit, (l / 8) % 2 the middle one, (l / 4) % 2 the lowest.
__device__ __forceinline__ float warp_sum8(float (&v)[8], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float send = lane & 16 ? v[i] : v[i + 4], mine = lane & 16 ? v[i + 4] : v[i];
    v[i] = mine + __shfl_xor_sync(0xffffffffu, send, 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float send = lane & 8 ? v[i] : v[i + 2], mine = lane & 8 ? v[i + 2] : v[i];
    v[i] = mine + __shfl_xor_sync(0xffffffffu, send, 8);
  }
  {
    const float send = lane & 4 ? v[0] : v[1], mine = lane & 4 ? v[1] : v[0];
    v[0] = mine + __shfl_xor_sync(0xffffffffu, send, 4);
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
  return v[0];
}

constexpr int kSums = 5;  // column sums: pre gamma, pre beta, gate, post gamma, post beta

// A block of `groups` groups of W warps, a row per group and step; a lane owns 8 G columns of every row
// that its group takes, so the column sums stay with it (G = 1: in registers, else in shared memory) and
// leave once per block, into partial[block][kSums][cols].
template <typename T, bool VEC, int G>
__global__ void __launch_bounds__(512, 1) block_norm_bwd_kernel(const BlockNormArgs a, int W, int groups,
                                                                float* __restrict__ partial) {
  extern __shared__ float shared_sums[];  // [kSums][cols]
  __shared__ float red[2][16][8];         // the two latest rows' sums of every warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / W, w = warp - group * W;
  const PhiloxState ps = philox_state(a.mask);
  const float inv_n = 1.f / (float)a.cols;
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr;
  float acc[G == 1 ? kSums : 1][8];
  if constexpr (G == 1) {
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;
  } else {
    for (int i = threadIdx.x; i < kSums * a.cols; i += blockDim.x) shared_sums[i] = 0.f;
    __syncthreads();
  }
  int flip = 0;
  for (long long row = (long long)blockIdx.x * groups + group; row < a.rows; row += (long long)gridDim.x * groups) {
    const size_t base = (size_t)row * a.cols;
    const float4 st = __ldg(reinterpret_cast<const float4*>(a.stats) + row);
    const float my = st.x, ry = st.y, mx = st.z, rx = st.w;
    float xh[G][8], e[G][8], yh[G][8], dh[G][8], c[G][8];
    uint32_t keep[G];
    float s[8] = {};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (g * W + w) * 256, left = a.cols - c0;
      float p[8];
      if (a.d_x_out) span_load<VEC>(a.d_x_out + base + c0, left, lane, e[g]);
      span_load<VEC>(static_cast<const T*>(a.y) + base + c0, left, lane, yh[g]);
      if (pre) {
        span_load<VEC>(a.x_out + base + c0, left, lane, xh[g]);
        span_load<VEC>(static_cast<const T*>(a.d_h) + base + c0, left, lane, dh[g]);
        span_load<VEC>(static_cast<const T*>(a.pre_gamma) + c0, left, lane, p);
      }
      keep[g] = span_keep<VEC>(a.mask, ps, (unsigned long long)row * ((a.cols + 7) / 8) + c0 / 8, lane);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool in = span_col<VEC>(lane, k) < left;
        if (!a.d_x_out) e[g][k] = 0.f;
        if (pre) {
          xh[g][k] = in ? (xh[g][k] - mx) * rx : 0.f;
          const float gg = dh[g][k] * p[k];
          s[0] += gg;
          s[1] = fmaf(gg, xh[g][k], s[1]);
          e[g][k] = fmaf(rx, gg, e[g][k]);
        } else {
          xh[g][k] = dh[g][k] = 0.f;
        }
        if (post) yh[g][k] = in ? (yh[g][k] - my) * ry : 0.f;
      }
      if (post) {
        span_load<VEC>(static_cast<const T*>(a.post_gamma) + c0, left, lane, c[g]);
        if (a.gate) {
          span_load<VEC>(static_cast<const T*>(a.gate) + (a.gate_rows ? base : 0) + c0, left, lane, p);
#pragma unroll
          for (int k = 0; k < 8; ++k) c[g][k] *= p[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          c[g][k] = keep[g] >> k & 1u ? c[g][k] * a.mask.scale : 0.f;
          const float ce = c[g][k] * e[g][k];
          s[2] += ce;
          s[3] += c[g][k];
          s[4] = fmaf(c[g][k], xh[g][k], s[4]);
          s[5] = fmaf(ce, yh[g][k], s[5]);
          s[6] = fmaf(c[g][k], yh[g][k], s[6]);
          s[7] = fmaf(c[g][k] * yh[g][k], xh[g][k], s[7]);
        }
      }
    }
    if (pre || post) {
      float total = warp_sum8(s, lane);
      if (W > 1) {
        if (lane % 4 == 0) red[flip][warp][lane / 4] = total;
        named_bar_sync(1 + group, 32 * W);
        total = 0.f;
        for (int i = lane & 3; i < W; i += 4) total += red[flip][group * W + i][lane / 4];
        total += __shfl_xor_sync(0xffffffffu, total, 2);
        total += __shfl_xor_sync(0xffffffffu, total, 1);
        flip ^= 1;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = __shfl_sync(0xffffffffu, total, 4 * i);
    }
    const float A = pre && !a.rms ? rx * s[0] * inv_n : 0.f, B = pre ? rx * s[1] * inv_n : 0.f;
    const float m0 = a.rms ? 0.f : (s[2] - A * s[3] - B * s[4]) * inv_n, m1 = (s[5] - A * s[6] - B * s[7]) * inv_n;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (g * W + w) * 256, left = a.cols - c0;
      float gate[8], gamma[8], beta[8], out[8], term[kSums][8];
      if (a.gate) span_load<VEC>(static_cast<const T*>(a.gate) + (a.gate_rows ? base : 0) + c0, left, lane, gate);
      if (post) span_load<VEC>(static_cast<const T*>(a.post_gamma) + c0, left, lane, gamma);
      if (a.post_beta) span_load<VEC>(static_cast<const T*>(a.post_beta) + c0, left, lane, beta);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float Gk = e[g][k] - A - xh[g][k] * B;
        out[k] = a.residual_scale * Gk;
        const float kept = keep[g] >> k & 1u ? Gk * a.mask.scale : 0.f;
        float n = yh[g][k];
        if (post) n = n * gamma[k] + (a.post_beta ? beta[k] : 0.f);
        const float dn = a.gate ? kept * gate[k] : kept;
        term[0][k] = dh[g][k] * xh[g][k];
        term[1][k] = dh[g][k];
        term[2][k] = keep[g] >> k & 1u ? kept * n : 0.f;
        term[3][k] = dn * yh[g][k];
        term[4][k] = dn;
        c[g][k] = post ? ry * (dn * gamma[k] - m0 - yh[g][k] * m1) : dn;
      }
      span_store<VEC>(a.dx + base + c0, left, lane, out);
      span_store<VEC>(static_cast<T*>(a.dy) + base + c0, left, lane, c[g]);
      if (a.gate_rows && a.d_gate) span_store<VEC>(static_cast<T*>(a.d_gate) + base + c0, left, lane, term[2]);
#pragma unroll
      for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (G == 1) acc[i][k] += term[i][k];
          else if (span_col<VEC>(lane, k) < left) shared_sums[(size_t)i * a.cols + c0 + span_col<VEC>(lane, k)] += term[i][k];
        }
    }
  }
  if constexpr (G == 1) {
    // the groups add their sums in order
    const int c0 = w * 256, left = a.cols - c0;
    for (int turn = 0; turn < groups; ++turn) {
      if (turn == group) {
#pragma unroll
        for (int i = 0; i < kSums; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int col = span_col<VEC>(lane, k);
            if (col < left) {
              float* at = shared_sums + (size_t)i * a.cols + c0 + col;
              *at = turn ? *at + acc[i][k] : acc[i][k];
            }
          }
      }
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kSums * a.cols; i += blockDim.x)
    partial[(size_t)blockIdx.x * kSums * a.cols + i] = shared_sums[i];
}

struct SumOutputs {
  float* out[kSums];
};

// out[i][c] = sum over the blocks of partial[block][i][c], in a fixed order: warp w of the block adds
// blocks w, w + 8, ..., then the warps' sums are added in order.
__global__ void __launch_bounds__(256) block_norm_sums_kernel(const float* __restrict__ partial, int blocks, int cols,
                                                              const SumOutputs o) {
  __shared__ float part[8][32];
  float* out = o.out[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols)
#pragma unroll 4
    for (int b = warp; b < blocks; b += 8) s += __ldg(partial + ((size_t)b * kSums + blockIdx.y) * cols + c);
  part[warp][lane] = s;
  __syncthreads();
  if (warp || c >= cols) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += part[i][lane];
  out[c] = s;
}

struct BwdShape {
  int G, W, groups, blocks;
};
BwdShape bwd_shape(int rows, int cols, int num_sms) {
  BwdShape s;
  const int spans = (cols + 255) / 256;
  s.G = spans > 16 ? 2 : 1;
  s.W = (spans + s.G - 1) / s.G;
  s.groups = s.G == 2 ? 1 : std::max(1, std::min(15, 16 / s.W));
  s.blocks = std::max(1, std::min(num_sms, (rows + s.groups - 1) / s.groups));
  return s;
}

template <typename T, bool VEC, int G>
cudaError_t launch_bwd(const BlockNormArgs& a, const BwdShape& s, float* partial, cudaStream_t st) {
  const size_t smem = sizeof(float) * kSums * a.cols;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(block_norm_bwd_kernel<T, VEC, G>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  block_norm_bwd_kernel<T, VEC, G><<<s.blocks, 32 * s.W * s.groups, smem, st>>>(a, s.W, s.groups, partial);
  return cudaGetLastError();
}

template <typename T, bool VEC>
void launch_fwd(const BlockNormArgs& a, cudaStream_t st) {
  const int spans = (a.cols + 255) / 256;
  const int W = (spans + 4) / 5, G = (spans + W - 1) / W;  // up to five spans per warp
  const int rows_per_block = W > 1 ? 1 : 4;
  const unsigned grid = (unsigned)((a.rows + rows_per_block - 1) / rows_per_block);
  const int threads = 32 * W * rows_per_block;
  switch (G) {
    case 1: block_norm_kernel<T, VEC, 1><<<grid, threads, 0, st>>>(a, W); break;
    case 2: block_norm_kernel<T, VEC, 2><<<grid, threads, 0, st>>>(a, W); break;
    case 3: block_norm_kernel<T, VEC, 3><<<grid, threads, 0, st>>>(a, W); break;
    case 4: block_norm_kernel<T, VEC, 4><<<grid, threads, 0, st>>>(a, W); break;
    default: block_norm_kernel<T, VEC, 5><<<grid, threads, 0, st>>>(a, W); break;
  }
}

// 16-byte accesses to every row and parameter
bool all_on_16(const BlockNormArgs& a, bool bf16) {
  const int es = bf16 ? 2 : 4, n = a.cols;
  return rows_on_16(a.y, n, es) && rows_on_16(a.x, n, 4) && rows_on_16(a.x_out, n, 4) && rows_on_16(a.h, n, es) &&
         rows_on_16(a.d_x_out, n, 4) && rows_on_16(a.d_h, n, es) && rows_on_16(a.dx, n, 4) && rows_on_16(a.dy, n, es) &&
         rows_on_16(a.post_gamma, n, es) && rows_on_16(a.post_beta, n, es) && rows_on_16(a.pre_gamma, n, es) &&
         rows_on_16(a.pre_beta, n, es) && rows_on_16(a.gate, n, es) &&
         (!a.gate_rows || rows_on_16(a.d_gate, n, es));
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const bool vec = all_on_16(a, bf16);
  if (bf16) {
    if (vec) launch_fwd<__nv_bfloat16, true>(a, st);
    else launch_fwd<__nv_bfloat16, false>(a, st);
  } else {
    if (vec) launch_fwd<float, true>(a, st);
    else launch_fwd<float, false>(a, st);
  }
  return cudaGetLastError();
}

size_t block_norm_bwd_workspace_bytes(int rows, int cols, int num_sms) {
  return sizeof(float) * kSums * (size_t)cols * bwd_shape(rows, cols, num_sms).blocks;
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, bool bf16, void* workspace, int num_sms, cudaStream_t st) {
  const BwdShape s = bwd_shape(a.rows, a.cols, num_sms);
  float* partial = static_cast<float*>(workspace);
  const bool vec = all_on_16(a, bf16);
  cudaError_t e;
  if (s.G == 1) {
    if (bf16) e = vec ? launch_bwd<__nv_bfloat16, true, 1>(a, s, partial, st) : launch_bwd<__nv_bfloat16, false, 1>(a, s, partial, st);
    else e = vec ? launch_bwd<float, true, 1>(a, s, partial, st) : launch_bwd<float, false, 1>(a, s, partial, st);
  } else {
    if (bf16) e = vec ? launch_bwd<__nv_bfloat16, true, 2>(a, s, partial, st) : launch_bwd<__nv_bfloat16, false, 2>(a, s, partial, st);
    else e = vec ? launch_bwd<float, true, 2>(a, s, partial, st) : launch_bwd<float, false, 2>(a, s, partial, st);
  }
  if (e != cudaSuccess) return e;
  SumOutputs o{{a.d_pre_gamma, a.d_pre_beta, a.gate_rows ? nullptr : static_cast<float*>(a.d_gate), a.d_post_gamma,
                a.d_post_beta}};
  block_norm_sums_kernel<<<dim3((a.cols + 31) / 32, kSums), 256, 0, st>>>(partial, s.blocks, a.cols, o);
  return cudaGetLastError();
}

}  // namespace esm
