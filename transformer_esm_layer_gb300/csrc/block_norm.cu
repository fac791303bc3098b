// The residual stream between two blocks, in one pass over it:
//   u = dropout(post(y)),  x_out = residual_scale * x + gate * u,  h = pre(x_out)
// post: the norm after the block that made y (or none); pre: the norm before the next block (or none);
// each a LayerNorm, (z - mean) / sqrt(var + eps) * gamma + beta with the biased variance, or an RMS norm,
// z / sqrt(mean(z^2) + eps) * gamma + beta.  And its gradient.
//
// Bound by memory: 12 bytes an element forward and 18 backward with bfloat16 blocks (the residual
// stream and its gradient are float32).  So every value is read and written once, a row's statistics and
// sums never leave the SM, and the rows to come are copied into shared memory while this one is worked on.
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

// Mean and 1 / sqrt(var + eps) of a row of `cols` values held by W warps, 256 columns each.  A warp's own
// mean and squared deviations are taken in two passes over its registers; those of several warps are
// joined with their counts (Chan, Golub, LeVeque 1979): no digits are lost to a large mean, and there
// is one barrier.  slot: [W] of shared memory; sync: the barrier of the row's threads.
template <bool VEC, typename Sync>
__device__ __forceinline__ float2 row_moments(const float (&z)[8], bool rms, float eps, int cols, int left, int W, int w,
                                              int lane, float2* slot, Sync sync) {
  float mean = 0.f, q = 0.f;
  if (!rms) {
    const float s = ((z[0] + z[1]) + (z[2] + z[3])) + ((z[4] + z[5]) + (z[6] + z[7]));
    mean = warp_sum(s) / (float)min(left, 256);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float d = span_col<VEC>(lane, k) < left ? z[k] - mean : 0.f;
    q = fmaf(d, d, q);
  }
  q = warp_sum(q);
  if (W > 1) {
    if (lane == 0) slot[w] = make_float2(mean, q);
    sync();
    const float last = (float)(cols - 256 * (W - 1));
    float m = 0.f;
    q = 0.f;
    if (!rms) {
      for (int i = 0; i < W - 1; ++i) m += slot[i].x;
      m = (m * 256.f + slot[W - 1].x * last) / (float)cols;
    }
    for (int i = 0; i < W; ++i) {
      const float2 o = slot[i];
      const float d = o.x - m;
      q += fmaf((i < W - 1 ? 256.f : last) * d, d, o.y);
    }
    mean = m;
  }
  return make_float2(mean, rsqrtf(q / (float)cols + eps));
}

// ---- forward ----
// One warp per 256 columns, W = ceil(cols / 256) warps per row and block; a block takes every gridDim.x-th
// row.  Some rows of x and y are on their way while one is worked on (VEC; rows that do not start
// on 16 bytes are read where they are used).
template <int MAXT>
constexpr int kFwdStages = MAXT <= 256 ? 4 : 3;  // (8192 float32 columns: 64 KB each)

template <typename T, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 4 : 1) block_norm_kernel(const BlockNormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 slots[2][2][32];
  const int W = blockDim.x >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = w * 256, left = a.cols - c0;
  const bool post_on = a.post_gamma != nullptr, pre_on = a.pre_gamma != nullptr;
  const size_t stage_bytes = (size_t)(2 + kChunks<T>) * blockDim.x * 16;
  const T* yc = static_cast<const T*>(a.y) + c0;
  const float* xc = a.x + c0;
  auto copy_ahead = [&](long long row, int stage) {
    if (row < a.rows) {
      stage_copy(ring + stage * stage_bytes, 0, xc + (size_t)row * a.cols, left, lane);
      stage_copy(ring + stage * stage_bytes, 2, yc + (size_t)row * a.cols, left, lane);
    }
    cp_async_commit();
  };
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kFwdStages<MAXT> - 1; ++i) copy_ahead(blockIdx.x + (long long)i * gridDim.x, i);
  }
  const PhiloxState ps = philox_state(a.mask);
  const int per_row = (a.cols + 7) / 8;
  // bfloat16 parameters stay in registers, float32 ones are read again for every row (from the L1)
  constexpr bool kKeep = sizeof(T) == 2 && VEC;
  Span8<T, VEC> post_gamma, post_beta, pre_gamma, pre_beta, gate;
  auto fetch = [&](Span8<T, VEC>& to, const void* p, float without) {
    to.fill(without);
    if (p) to.load(static_cast<const T*>(p) + c0, left, lane);
  };
  if (kKeep) {
    fetch(post_gamma, a.post_gamma, 1.f);
    fetch(post_beta, a.post_beta, 0.f);
    fetch(pre_gamma, a.pre_gamma, 1.f);
    fetch(pre_beta, a.pre_beta, 0.f);
    if (!a.gate_rows) fetch(gate, a.gate, 1.f);
  }
  int stage = 0, flip = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = (size_t)row * a.cols + c0;
    float x[8], u[8], p[8];
    if (a.gate_rows) gate.load(static_cast<const T*>(a.gate) + base, left, lane);
    if constexpr (VEC) {
      copy_ahead(row + (long long)(kFwdStages<MAXT> - 1) * gridDim.x, stage == 0 ? kFwdStages<MAXT> - 1 : stage - 1);
      cp_async_wait<kFwdStages<MAXT> - 1>();
      stage_read<float>(ring + stage * stage_bytes, 0, x);
      stage_read<T>(ring + stage * stage_bytes, 2, u);
      stage = stage == kFwdStages<MAXT> - 1 ? 0 : stage + 1;
    } else {
      span_load<VEC>(xc + (size_t)row * a.cols, left, lane, x);
      span_load<VEC>(yc + (size_t)row * a.cols, left, lane, u);
    }
    float2 post = make_float2(0.f, 0.f), pre = make_float2(0.f, 0.f);
    const uint32_t keep = span_keep<VEC>(a.mask, ps, (unsigned long long)row * per_row + c0 / 8, lane);
    if (post_on) {
      post = row_moments<VEC>(u, a.rms, a.eps, a.cols, left, W, w, lane, slots[flip][0], [] { __syncthreads(); });
      float b[8];
      if (!kKeep) {
        fetch(post_gamma, a.post_gamma, 1.f);
        fetch(post_beta, a.post_beta, 0.f);
      }
      post_gamma.get(p);
      post_beta.get(b);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = fmaf((u[k] - post.x) * post.y, p[k], b[k]);
    }
    if (!kKeep && !a.gate_rows) fetch(gate, a.gate, 1.f);
    gate.get(p);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = keep >> k & 1u ? u[k] * a.mask.scale : 0.f;
      x[k] = fmaf(a.residual_scale, x[k], p[k] * v);
    }
    span_store<VEC>(a.x_out + base, left, lane, x);
    if (pre_on) {
      float b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = span_col<VEC>(lane, k) < left ? x[k] : 0.f;
      pre = row_moments<VEC>(x, a.rms, a.eps, a.cols, left, W, w, lane, slots[flip][1], [] { __syncthreads(); });
      if (!kKeep) {
        fetch(pre_gamma, a.pre_gamma, 1.f);
        fetch(pre_beta, a.pre_beta, 0.f);
      }
      pre_gamma.get(p);
      pre_beta.get(b);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = fmaf((x[k] - pre.x) * pre.y, p[k], b[k]);
      span_store<VEC>(static_cast<T*>(a.h) + base, left, lane, x);
    }
    if (a.stats && threadIdx.x == 0)
      reinterpret_cast<float4*>(a.stats)[row] = make_float4(post.x, post.y, pre.x, pre.y);
    flip ^= 1;
  }
}

// ---- backward ----
// With xh = (x_out - mean) rstd, yh likewise, k = keep * scale * gate, g = d_h * gamma_pre:
//   G  = d_x_out + rstd_x (g - mean(g) - xh mean(g xh))        dx = residual_scale G
//   u's gradient, through gate and dropout, is k G, and with c = k gamma_post
//   dy = rstd_y (c G - mean(c G) - yh mean(c G yh))
// The means over c G hold G, which holds the means over g; but G is linear in those, so with
// e = d_x_out + rstd_x g all of a row's sums
//   S0 = sum g, S1 = sum g xh, S2 = sum c e, S3 = sum c, S4 = sum c xh, S5 = sum c yh e, S6 = sum c yh,
//   S7 = sum c yh xh
// are taken in one exchange:  sum c G = S2 - rstd_x (S0 S3 + S1 S4) / cols, and so on.
// The parameters' gradients come of four column sums: d_h xh, d_h, and with q = keep scale G
//   P = sum q yh, Q = sum q:  dgate = gamma_post P + beta_post Q, dgamma_post = gate P, dbeta_post = gate Q
// (a gate of its own for every row goes into q instead, and its gradient is written row by row).
//
// Eight sums over a warp: every step halves the number of values that a lane still adds, and lanes 4 i to
// 4 i + 3 end with the total of value i.
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
  const float send = lane & 4 ? v[0] : v[1], mine = lane & 4 ? v[1] : v[0];
  float total = mine + __shfl_xor_sync(0xffffffffu, send, 4);
  total += __shfl_xor_sync(0xffffffffu, total, 2);
  total += __shfl_xor_sync(0xffffffffu, total, 1);
  return total;
}

constexpr int kSums = 4;         // column sums: d_h xh, d_h, P, Q
constexpr int kBwdWarps = 20;    // warps of a block

// A block of `groups` groups of W warps, a row per group and step; a lane owns 8 G columns of every row
// that its group takes, so the column sums stay with it (G = 1: in registers, else in shared memory) and
// leave once per block, into partial[block][kSums][cols].
template <typename T, bool VEC, int G, int STAGES>
__global__ void __launch_bounds__(G == 1 ? 32 * kBwdWarps : 512, 1)
    block_norm_bwd_kernel(const BlockNormArgs a, int W, int groups, float* __restrict__ partial) {
  extern __shared__ __align__(16) uint8_t smem[];  // the stages of copies ahead; [kSums][cols] sums
  __shared__ float red[2][kBwdWarps][8];           // the two latest rows' sums of every warp
  float* sums = reinterpret_cast<float*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / W, w = warp - group * W;
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr;
  const long long first = (long long)blockIdx.x * groups + group, step = (long long)gridDim.x * groups;
  // chunks of a stage: d_x_out, y, x_out, d_h, the gate's row
  constexpr int cy = 2, cx = cy + kChunks<T>, ch = cx + 2, cg = ch + kChunks<T>;
  const size_t stage_bytes = (size_t)(cg + (a.gate_rows ? kChunks<T> : 0)) * blockDim.x * 16;
  auto copy_ahead = [&](long long row, int stage) {
    if (row < a.rows) {
      uint8_t* at = smem + stage * stage_bytes;
      const size_t base = (size_t)row * a.cols + w * 256;
      const int left = a.cols - w * 256;
      if (a.d_x_out) stage_copy(at, 0, a.d_x_out + base, left, lane);
      stage_copy(at, cy, static_cast<const T*>(a.y) + base, left, lane);
      if (pre) {
        stage_copy(at, cx, static_cast<const float*>(a.x_out) + base, left, lane);
        stage_copy(at, ch, static_cast<const T*>(a.d_h) + base, left, lane);
      }
      if (a.gate_rows) stage_copy(at, cg, static_cast<const T*>(a.gate) + base, left, lane);
    }
    cp_async_commit();
  };
  if constexpr (STAGES > 0) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) copy_ahead(first + i * step, i);
  }
  const PhiloxState ps = philox_state(a.mask);
  const float inv_n = 1.f / (float)a.cols;
  const int per_row = (a.cols + 7) / 8;
  float acc[G == 1 ? kSums : 1][8];
  if constexpr (G == 1) {
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;
  } else {
    for (int i = threadIdx.x; i < kSums * a.cols; i += blockDim.x) sums[i] = 0.f;
    __syncthreads();
  }
  int flip = 0, stage = 0;
  for (long long row = first; row < a.rows; row += step) {
    const float4 st = pre || post ? __ldg(reinterpret_cast<const float4*>(a.stats) + row) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float my = st.x, ry = st.y, mx = st.z, rx = st.w;
    const uint8_t* at = smem + stage * stage_bytes;
    if constexpr (STAGES > 0) {
      copy_ahead(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
      cp_async_wait<STAGES - 1>();
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    float xh[G][8], e[G][8], yh[G][8], c[G][8];
    uint32_t keep[G];
    float s[8] = {};
    auto add = [&](int g, int i, int k, float v) {
      if constexpr (G == 1) {
        acc[i][k] += v;
      } else {
        const int col = (g * W + w) * 256 + span_col<VEC>(lane, k);
        if (col < a.cols) sums[(size_t)i * a.cols + col] += v;
      }
    };
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (g * W + w) * 256, left = a.cols - c0;
      const size_t base = (size_t)row * a.cols + c0;
      float dh[8], p[8];
      if constexpr (STAGES > 0) {
        stage_read<float>(at, 0, e[g]);
        stage_read<T>(at, cy, yh[g]);
        stage_read<float>(at, cx, xh[g]);
        stage_read<T>(at, ch, dh);
      } else {
        if (a.d_x_out) span_load<VEC>(a.d_x_out + base, left, lane, e[g]);
        span_load<VEC>(static_cast<const T*>(a.y) + base, left, lane, yh[g]);
        if (pre) {
          span_load<VEC>(static_cast<const float*>(a.x_out) + base, left, lane, xh[g]);
          span_load<VEC>(static_cast<const T*>(a.d_h) + base, left, lane, dh);
        }
      }
      if (!a.d_x_out) {
#pragma unroll
        for (int k = 0; k < 8; ++k) e[g][k] = 0.f;
      }
      keep[g] = span_keep<VEC>(a.mask, ps, (unsigned long long)row * per_row + c0 / 8, lane);
      if (pre) {
        Span8<T, VEC> gamma;
        gamma.load(static_cast<const T*>(a.pre_gamma) + c0, left, lane);
        gamma.get(p);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          xh[g][k] = span_col<VEC>(lane, k) < left ? (xh[g][k] - mx) * rx : 0.f;
          const float gg = dh[k] * p[k];
          add(g, 0, k, dh[k] * xh[g][k]);
          add(g, 1, k, dh[k]);
          s[0] += gg;
          s[1] = fmaf(gg, xh[g][k], s[1]);
          e[g][k] = fmaf(rx, gg, e[g][k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) xh[g][k] = 0.f;
      }
      if (post) {
        Span8<T, VEC> gamma;
        gamma.load(static_cast<const T*>(a.post_gamma) + c0, left, lane);
        gamma.get(c[g]);
        if (a.gate) {
          if (STAGES > 0 && a.gate_rows) {
            stage_read<T>(at, cg, p);
          } else {
            gamma.load(static_cast<const T*>(a.gate) + (a.gate_rows ? base : c0), left, lane);
            gamma.get(p);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) c[g][k] *= p[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          yh[g][k] = span_col<VEC>(lane, k) < left ? (yh[g][k] - my) * ry : 0.f;
          c[g][k] = keep[g] >> k & 1u ? c[g][k] * a.mask.scale : 0.f;
          const float ce = c[g][k] * e[g][k], cyh = c[g][k] * yh[g][k];
          s[2] += ce;
          s[3] += c[g][k];
          s[4] = fmaf(c[g][k], xh[g][k], s[4]);
          s[5] = fmaf(ce, yh[g][k], s[5]);
          s[6] += cyh;
          s[7] = fmaf(cyh, xh[g][k], s[7]);
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
      const size_t base = (size_t)row * a.cols + c0;
      float out[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        e[g][k] = fmaf(-B, xh[g][k], e[g][k] - A);  // now G
        out[k] = a.residual_scale * e[g][k];
      }
      span_store<VEC>(a.dx + base, left, lane, out);
      if (a.gate_rows) {
        float gate[8], n[8];
        if constexpr (STAGES > 0) stage_read<T>(at, cg, gate);
        else span_load<VEC>(static_cast<const T*>(a.gate) + base, left, lane, gate);
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k] = yh[g][k];
        if (post) {
          float p[8];
          Span8<T, VEC> v;
          v.load(static_cast<const T*>(a.post_gamma) + c0, left, lane);
          v.get(p);
#pragma unroll
          for (int k = 0; k < 8; ++k) n[k] *= p[k];
          if (a.post_beta) {
            v.load(static_cast<const T*>(a.post_beta) + c0, left, lane);
            v.get(p);
#pragma unroll
            for (int k = 0; k < 8; ++k) n[k] += p[k];
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool kept = keep[g] >> k & 1u;
          const float q = kept ? e[g][k] * a.mask.scale : 0.f;
          n[k] = kept ? q * n[k] : 0.f;
          out[k] = q * gate[k];
        }
        if (a.d_gate) span_store<VEC>(static_cast<T*>(a.d_gate) + base, left, lane, n);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] = keep[g] >> k & 1u ? e[g][k] * a.mask.scale : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // (a dropped value adds nothing, whatever y holds there)
        add(g, 2, k, keep[g] >> k & 1u ? out[k] * yh[g][k] : 0.f);
        add(g, 3, k, out[k]);
      }
      if (post) {
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] = ry * (fmaf(c[g][k], e[g][k], -m0) - yh[g][k] * m1);
      } else if (a.gate && !a.gate_rows) {
        float p[8];
        Span8<T, VEC> v;
        v.load(static_cast<const T*>(a.gate) + c0, left, lane);
        v.get(p);
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] *= p[k];
      }
      span_store<VEC>(static_cast<T*>(a.dy) + base, left, lane, out);
    }
  }
  if constexpr (G == 1) {
    // the stages' place is taken by the sums, which the groups add in order
    if constexpr (STAGES > 0) cp_async_wait<0>();
    __syncthreads();
    const int c0 = w * 256, left = a.cols - c0;
    for (int turn = 0; turn < groups; ++turn) {
      if (turn == group) {
#pragma unroll
        for (int i = 0; i < kSums; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int col = span_col<VEC>(lane, k);
            if (col < left) {
              float* to = sums + (size_t)i * a.cols + c0 + col;
              *to = turn ? *to + acc[i][k] : acc[i][k];
            }
          }
      }
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kSums * a.cols; i += blockDim.x)
    partial[(size_t)blockIdx.x * kSums * a.cols + i] = sums[i];
}

// The parameters' gradients from the blocks' column sums, in a fixed order: warp w of a block adds blocks
// w, w + 16, ... of 32 columns, then the warps' sums are added in order.  blockIdx.y: the sums of pre, of post.
template <typename T>
__global__ void __launch_bounds__(512) block_norm_sums_kernel(const BlockNormArgs a, const float* __restrict__ partial,
                                                              int blocks) {
  __shared__ float part[2][16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, post = blockIdx.y;
  float s0 = 0.f, s1 = 0.f;
  if (c < a.cols) {
#pragma unroll 4
    for (int b = warp; b < blocks; b += 16) {
      const float* at = partial + ((size_t)b * kSums + 2 * post) * a.cols + c;
      s0 += __ldg(at);
      s1 += __ldg(at + a.cols);
    }
  }
  part[0][warp][lane] = s0;
  part[1][warp][lane] = s1;
  __syncthreads();
  if (warp || c >= a.cols) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    s0 += part[0][i][lane];
    s1 += part[1][i][lane];
  }
  if (!post) {
    if (a.d_pre_gamma) a.d_pre_gamma[c] = s0;
    if (a.d_pre_beta) a.d_pre_beta[c] = s1;
    return;
  }
  const bool vector = a.gate && !a.gate_rows;
  const float gate = vector ? ld1(static_cast<const T*>(a.gate) + c) : 1.f;
  if (a.d_post_gamma) a.d_post_gamma[c] = gate * s0;
  if (a.d_post_beta) a.d_post_beta[c] = gate * s1;
  if (vector && a.d_gate) {
    float g = s0;
    if (a.post_gamma) g *= ld1(static_cast<const T*>(a.post_gamma) + c);
    if (a.post_beta) g = fmaf(ld1(static_cast<const T*>(a.post_beta) + c), s1, g);
    static_cast<float*>(a.d_gate)[c] = g;
  }
}

struct BwdShape {
  int G, W, groups, blocks;
};
BwdShape bwd_shape(int rows, int cols, int num_sms) {
  BwdShape s;
  const int spans = (cols + 255) / 256;
  s.G = spans > 16 ? 2 : 1;
  s.W = (spans + s.G - 1) / s.G;
  s.groups = s.G == 2 ? 1 : std::min(15, kBwdWarps / s.W);
  s.blocks = std::max(1, std::min(num_sms, (rows + s.groups - 1) / s.groups));
  return s;
}

constexpr size_t kSmemMax = 227 * 1024 - 2048;  // (the rest: static shared memory)

template <typename T, bool VEC, int G, int STAGES>
cudaError_t launch_bwd_as(const BlockNormArgs& a, const BwdShape& s, size_t stage, float* partial, cudaStream_t st) {
  const size_t smem = std::max(sizeof(float) * kSums * a.cols, stage * STAGES);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(block_norm_bwd_kernel<T, VEC, G, STAGES>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  block_norm_bwd_kernel<T, VEC, G, STAGES><<<s.blocks, 32 * s.W * s.groups, smem, st>>>(a, s.W, s.groups, partial);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const BlockNormArgs& a, bool vec, float* partial, int num_sms, cudaStream_t st) {
  const BwdShape s = bwd_shape(a.rows, a.cols, num_sms);
  const size_t stage = (size_t)(4 + (a.gate_rows ? 3 : 2) * kChunks<T>) * 16 * 32 * s.W * s.groups;
  cudaError_t e;
  if (s.G == 2) e = vec ? launch_bwd_as<T, true, 2, 0>(a, s, 0, partial, st) : launch_bwd_as<T, false, 2, 0>(a, s, 0, partial, st);
  else if (!vec) e = launch_bwd_as<T, false, 1, 0>(a, s, 0, partial, st);
  else if (3 * stage <= kSmemMax) e = launch_bwd_as<T, true, 1, 3>(a, s, stage, partial, st);
  else e = launch_bwd_as<T, true, 1, 2>(a, s, stage, partial, st);
  if (e != cudaSuccess) return e;
  block_norm_sums_kernel<T><<<dim3((a.cols + 31) / 32, 2), 512, 0, st>>>(a, partial, s.blocks);
  return cudaGetLastError();
}

template <typename T, bool VEC, int MAXT>
cudaError_t launch_fwd_as(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  const int threads = (a.cols + 255) / 256 * 32;
  const size_t smem = VEC ? (size_t)kFwdStages<MAXT> * (2 + kChunks<T>) * threads * 16 : 0;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(block_norm_kernel<T, VEC, MAXT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  // as many blocks as the SMs hold at once (64 registers per thread)
  const int per_sm = std::max(1, (int)std::min({(size_t)32, (size_t)1024 / threads, kSmemMax / (smem + 2048)}));
  const unsigned grid = (unsigned)std::min((long long)a.rows, (long long)num_sms * per_sm);
  block_norm_kernel<T, VEC, MAXT><<<grid, threads, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_fwd(const BlockNormArgs& a, bool vec, int num_sms, cudaStream_t st) {
  if (a.cols <= 2048)
    return vec ? launch_fwd_as<T, true, 256>(a, num_sms, st) : launch_fwd_as<T, false, 256>(a, num_sms, st);
  return vec ? launch_fwd_as<T, true, 1024>(a, num_sms, st) : launch_fwd_as<T, false, 1024>(a, num_sms, st);
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
  return bf16 ? launch_fwd<__nv_bfloat16>(a, vec, num_sms, st) : launch_fwd<float>(a, vec, num_sms, st);
}

size_t block_norm_bwd_workspace_bytes(int rows, int cols, int num_sms) {
  return sizeof(float) * kSums * (size_t)cols * bwd_shape(rows, cols, num_sms).blocks;
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, bool bf16, void* workspace, int num_sms, cudaStream_t st) {
  const bool vec = all_on_16(a, bf16);
  float* partial = static_cast<float*>(workspace);
  return bf16 ? launch_bwd<__nv_bfloat16>(a, vec, partial, num_sms, st) : launch_bwd<float>(a, vec, partial, num_sms, st);
}

}  // namespace esm
