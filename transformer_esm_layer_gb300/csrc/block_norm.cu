// The residual stream between two blocks, in one pass over it:
//   u = dropout(post(y)),  x_out = residual_scale * x + gate * u,  h = pre(x_out)
// post: the norm after the block that made y (or none); pre: the norm before the next block (or none);
// each a LayerNorm, (z - mean) / sqrt(var + eps) * gamma + beta with the biased variance, or an RMS norm,
// z / sqrt(mean(z^2) + eps) * gamma + beta.  And its gradient.
//
// Bound by memory: 12 bytes an element forward and 18 backward with bfloat16 blocks (the residual
// stream and its gradient are float32).  So every value is read and written once, a row's statistics and
// sums never leave the SM.  16384 x 1280 with two LayerNorms, gate and dropout: forward 46.3 us, 5.4 TB/s (the same
// five streams copied without arithmetic: 39.5 us), backward 73.7 us, 5.1 TB/s; without the dropout 44.3 and 68: the
// instructions of masks, sums and statistics are what keeps them off the memory's rate.
#include <algorithm>
#include <type_traits>

#include "dropout.cuh"
#include "internal.h"

namespace esm {
namespace {

// ---- forward ----
// A block takes R rows, W warps to each; a warp holds G spans of 256 columns, eight of each to a lane.  Rows
// come as blocks of the grid, not in a loop: the launch bounds keep 21 to 25 warps on the SM (14 to 20 with float32
// blocks), whose loads, sums and stores interleave by themselves (blocks that stay, with rows copied ahead by the
// threads, took 60 us where this took 49.5).
// Up to 2048 columns G = 1, and R = 2 where there are rows enough: the parameters are read and unpacked once
// for both, the generator's round keys are shared, and one barrier serves both rows' sums.
struct RowShape {
  float inv_cols, last, inv_last;  // of the columns of a row's last warp
};

// A warp's own mean and squared deviations are taken in two passes over its registers, and those of
// several warps joined by their counts (Chan, Golub, LeVeque 1979), so no digits are lost to a large mean
// and the row's warps meet once.  Counts are 256 G but for the last warp's; means are taken relative to the
// first warp's, so that one pass over the slots is enough:  sum of n d^2 about the joint mean is
// sum of n d^2 - cols shift^2.
template <int W, int G>
__device__ __forceinline__ float2 join_moments(const float2* slot, int warps, const RowShape& s) {
  const float2 first = slot[0];
  float d1 = 0.f, d2 = 0.f, q = first.y;
  auto add = [&](int i) {
    const float2 o = slot[i];
    const float d = o.x - first.x;
    d1 += d;
    d2 = fmaf(d, d, d2);
    q += o.y;
  };
  if constexpr (W > 0) {
#pragma unroll
    for (int i = 1; i < W - 1; ++i) add(i);
  } else {
#pragma unroll 4
    for (int i = 1; i < warps - 1; ++i) add(i);
  }
  const float2 o = slot[warps - 1];
  const float d = o.x - first.x, nd = s.last * d;
  d1 = fmaf(256.f * G, d1, nd);
  d2 = fmaf(256.f * G, d2, nd * d);
  const float shift = d1 * s.inv_cols;
  return make_float2(first.x + shift, q + o.y + fmaf(-shift, d1, d2));
}

// Mean and 1 / sqrt(var + eps) of R rows of which this lane holds z (0 past the row's end); left: columns from the
// warp's first on.
template <int R, int G, int W, bool VEC>
__device__ __forceinline__ void row_moments(const Pairs (&z)[R][G], const BlockNormArgs& a, const RowShape& s, int left,
                                            int warps, int w, int lane, float2 (*slot)[W > 0 ? W : 32], float2 (&out)[R]) {
  float mean[R], q[R];
#pragma unroll
  for (int r = 0; r < R; ++r) mean[r] = 0.f;
  if (!a.rms) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = sum(z[r][0]);
#pragma unroll
      for (int g = 1; g < G; ++g) mean[r] += sum(z[r][g]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) mean[r] += __shfl_xor_sync(0xffffffffu, mean[r], o);
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] *= w == warps - 1 ? s.inv_last : 1.f / (256.f * G);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint64_t t = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      Pairs d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = f2_add(z[r][g][i], f2_both(-mean[r]));
      if (left < 256 * (g + 1)) span_trim<VEC>(left - 256 * g, lane, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) t = g + i ? f2_fma(d[i], d[i], t) : f2_mul(d[0], d[0]);
    }
    q[r] = f2_sum(t);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int r = 0; r < R; ++r) q[r] += __shfl_xor_sync(0xffffffffu, q[r], o);
  if (warps > 1) {
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) slot[r][w] = make_float2(mean[r], q[r]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 j = make_float2(mean[r], q[r]);
    if (warps > 1) j = join_moments<W, G>(slot[r], warps, s);
    out[r] = make_float2(j.x, rsqrtf(fmaf(j.y, s.inv_cols, a.eps)));
  }
}

// W = 0: the number of warps is blockDim.x / 32.  VEC: every row's eights aligned and cols % 8 == 0.
template <typename T, bool VEC, int W, int R, int G, int MAX_THREADS, int MIN_BLOCKS>
__global__ void __launch_bounds__(MAX_THREADS, MIN_BLOCKS)
    block_norm_kernel(const BlockNormArgs a, const RowShape shape) {
  __shared__ float2 slots[2][R][W > 0 ? W : 32];
  const int warps = W > 0 ? W : blockDim.x >> 5, w = W == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int left = a.cols - w * G * 256;  // columns from the warp's first on
  using RawT = std::conditional_t<VEC, Raw8<T>, Pairs>;
  using RawF = std::conditional_t<VEC, Raw8<float>, Pairs>;
  // VEC: the lane's first column of each span, or, past the row's end, the row's first, and then it writes nothing
  bool active[G];
  int c[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (w * G + g) * 256;
    active[g] = 8 * lane < left - 256 * g;
    c[g] = VEC ? (active[g] ? c0 + 8 * lane : 0) : c0;
  }
  auto fetch = [&](auto* p, int g, auto& raw) {
    if constexpr (VEC) raw.load(p + c[g], 8);
    else span_load<false>(p + c[g], a.cols - c[g], lane, raw);
  };
  auto read = [](const auto& raw, Pairs& v) {
    if constexpr (VEC) raw.get(v);
    else v[0] = raw[0], v[1] = raw[1], v[2] = raw[2], v[3] = raw[3];
  };
  auto store = [&](auto* p, int g, const Pairs& v) {
    if constexpr (VEC) {
      if (active[g]) st8(p + c[g], v);
    } else {
      span_store<false>(p + c[g], a.cols - c[g], lane, v);
    }
  };
  auto trim = [&](Pairs (&v)[R][G]) {
    if (left < 256 * G) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int g = 0; g < G; ++g) span_trim<VEC>(left - 256 * g, lane, v[r][g]);
    }
  };
  // (an odd last row is worked on twice by a block of two, and written once)
  long long row[R];
  size_t base[R];
  RawT y[R][G], gate[R][G];
  RawF x[R][G];
  bool own[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const long long n = (long long)blockIdx.x * R + r;
    own[r] = n < a.rows;
    row[r] = own[r] ? n : a.rows - 1;
    base[r] = (size_t)row[r] * (uint32_t)a.cols;
#pragma unroll
    for (int g = 0; g < G; ++g) fetch(static_cast<const T*>(a.y) + base[r], g, y[r][g]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int g = 0; g < G; ++g) fetch(a.x + base[r], g, x[r][g]);
  if (a.gate_rows) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int g = 0; g < G; ++g) fetch(static_cast<const T*>(a.gate) + base[r], g, gate[r][g]);
  }
  uint4 words[R][G];
  const PhiloxState ps = philox_state(a.mask);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t block = (uint32_t)c[g] / 8 + (VEC ? 0 : lane);
      words[r][g] = drop_words(a.mask, ps, (unsigned long long)row[r] * ((uint32_t)(a.cols + 7) / 8) + block);
      words[r][g] = span_words<VEC>(a.mask, words[r][g], lane);
    }
  Pairs u[R][G], p;
  float2 post[R], pre[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int g = 0; g < G; ++g) read(y[r][g], u[r][g]);
    post[r] = pre[r] = make_float2(0.f, 0.f);
  }
  trim(u);
  auto vector = [&](const void* from, int g) {
    RawT raw;
    fetch(static_cast<const T*>(from), g, raw);
    read(raw, p);
  };
  auto normalise = [&](const float2 (&m)[R], const void* gamma, const void* beta) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      vector(gamma, g);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[r][g][i] = f2_mul(f2_mul(f2_add(u[r][g][i], f2_both(-m[r].x)), f2_both(m[r].y)), p[i]);
      if (beta) {
        vector(beta, g);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) u[r][g][i] = f2_add(u[r][g][i], p[i]);
      }
    }
  };
  if (a.post_gamma) {
    row_moments<R, G, W, VEC>(u, a, shape, left, warps, w, lane, slots[0], post);
    normalise(post, a.post_gamma, a.post_beta);
  }
  if (a.mask.rng) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[r][g][i] = f2_mul(u[r][g][i], f2_both(a.mask.scale));
        keep(words[r][g], ps, u[r][g]);
      }
  }
  if (a.gate) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!a.gate_rows) vector(a.gate, g);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (a.gate_rows) read(gate[r][g], p);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[r][g][i] = f2_mul(u[r][g][i], p[i]);
      }
    }
  }
  // (x_out may be x: a lane writes only places that it alone reads, and has read, a last row's twice)
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      read(x[r][g], p);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[r][g][i] = f2_fma(f2_both(a.residual_scale), p[i], u[r][g][i]);
      if (own[r]) store(a.x_out + base[r], g, u[r][g]);
    }
  if (a.pre_gamma) {
    trim(u);
    row_moments<R, G, W, VEC>(u, a, shape, left, warps, w, lane, slots[1], pre);
    normalise(pre, a.pre_gamma, a.pre_beta);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (own[r]) store(static_cast<T*>(a.h) + base[r], g, u[r][g]);
  }
  if (a.stats && threadIdx.x == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (own[r]) reinterpret_cast<float4*>(a.stats)[row[r]] = make_float4(post[r].x, post[r].y, pre[r].x, pre[r].y);
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
// (S1, S5 and S7 for an RMS norm) are taken in one exchange:  sum c G = S2 - rstd_x (S0 S3 + S1 S4) / cols, and so on.
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

// Four sums: lanes 8 i to 8 i + 7 end with the total of value i.
__device__ __forceinline__ float warp_sum4(float (&v)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float send = lane & 16 ? v[i] : v[i + 2], mine = lane & 16 ? v[i + 2] : v[i];
    v[i] = mine + __shfl_xor_sync(0xffffffffu, send, 16);
  }
  const float send = lane & 8 ? v[0] : v[1], mine = lane & 8 ? v[1] : v[0];
  float total = mine + __shfl_xor_sync(0xffffffffu, send, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  return total;
}

constexpr int kSums = 4;        // column sums: d_h xh, d_h, P, Q
constexpr int kBwdWarps = 20;   // warps of a block at most
constexpr int kStages = 2;      // rows of a group on their way (three were no faster)
constexpr int kMaxGroups = 15;  // named barriers
// The same with blocks of T: 96 registers are enough for bfloat16 ones (16384 x 1280: 73.7 us, 16 warps 81), float32 ones
// spill (84.8 us with 16 warps and 128 registers, 117 with 20).
template <typename T>
constexpr int kWarpsOf = sizeof(T) == 2 ? kBwdWarps : 16;

// Aligned eights, cols % 8 == 0 and a group's rows and sums in shared memory: cols <= 4096, float32 <= 4088 (at 4096 the
// kernel below: 5120 rows 131 us; 5130 of 4088 columns by this one 99).  A block of `groups` groups of
// W = ceil(cols / 256) warps stays on its SM and takes a row per group and step; a lane owns eight columns of every row
// that its group takes, so the four column sums stay with it (in shared memory, which frees 32 registers) and leave
// once per block, into partial[block][kSums][cols].  The rows to come arrive by bulk copies, kStages of them per
// group, which leaves the threads and the L1 out of it; gamma_pre and scale gate gamma_post stand in shared
// memory as float32.
template <typename T, bool RMS>
__global__ void __launch_bounds__(32 * kWarpsOf<T>, 1)
    block_norm_bwd_kernel(const BlockNormArgs a, int W, int groups, float* __restrict__ partial) {
  extern __shared__ __align__(16) uint8_t smem[];  // vectors, column sums, the rows on their way
  __shared__ float red[2][kBwdWarps][8];           // the two latest rows' sums of every warp
  __shared__ uint64_t full[kMaxGroups * kStages];
  __shared__ PhiloxKeys keys;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / W, w = warp - group * W;
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr, partly = a.cols - w * 256 < 256;
  const int c = w * 256 + 8 * lane;  // the lane's first column
  const bool active = c < a.cols;
  const int first = blockIdx.x * groups + group, step = gridDim.x * groups;  // (rows + 4 steps fit 32 bits)
  const PhiloxState ps = philox_state(a.mask);
  philox_keys(ps, &keys);
  // a stage: the statistics, rows of d_x_out and x_out (float32), of y and d_h (T)
  const uint32_t f_bytes = (uint32_t)a.cols * 4, t_bytes = (uint32_t)a.cols * sizeof(T);
  const uint32_t stage_bytes = 16 + 2 * f_bytes + 2 * t_bytes;
  // sum i of the lane's columns: its own 16 bytes at 2 i and 2 i + 1 blocks' widths
  float4* own_sums = reinterpret_cast<float4*>(smem + 2048 * W) + threadIdx.x;
  uint8_t* ring = smem + 2048 * W + (size_t)blockDim.x * (32 * kSums) + group * kStages * stage_bytes;
  uint64_t* bars = full + group * kStages;
  if (threadIdx.x < groups * kStages) mbar_init(full + threadIdx.x, 1);
  fence_barrier_init();
  bool alive = true;
  auto arrive = [&](int row, int stage) {  // (one thread of the group)
    if (row >= a.rows || !alive) return;
    const size_t at = (size_t)row * a.cols;
    uint8_t* to = ring + stage * stage_bytes;
    mbar_arrive_expect_tx(bars + stage, (pre || post ? 16 : 0) + (a.d_x_out ? f_bytes : 0) + t_bytes +
                                            (pre ? f_bytes + t_bytes : 0));
    if (pre || post) bulk_load(to, a.stats + 4 * (size_t)row, 16, bars + stage);
    to += 16;
    if (a.d_x_out) bulk_load(to, a.d_x_out + at, f_bytes, bars + stage);
    if (pre) bulk_load(to + f_bytes, a.x_out + at, f_bytes, bars + stage);
    to += 2 * f_bytes;
    bulk_load(to, static_cast<const T*>(a.y) + at, t_bytes, bars + stage);
    if (pre) bulk_load(to + t_bytes, static_cast<const T*>(a.d_h) + at, t_bytes, bars + stage);
  };
  __syncthreads();
  grid_dependency_launch();
  if (w == 0 && lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) arrive(first + i * step, i);
  }
  if (!a.d_x_out) {  // zeros stand in its place
    for (int s = 0; s < kStages; ++s)
      for (int i = w * 32 + lane; i < a.cols; i += 32 * W) reinterpret_cast<float*>(ring + 16 + s * stage_bytes)[i] = 0.f;
  }
  float* vf = reinterpret_cast<float*>(smem);
  for (int i = threadIdx.x; i < 256 * W; i += blockDim.x) {
    const int at = ((i >> 8) * 2 + (i >> 2 & 1)) * 128 + (i >> 3 & 31) * 4 + (i & 3);
    auto value = [&](const void* p, float without) { return p ? ld1(static_cast<const T*>(p) + i) : without; };
    vf[at] = i < a.cols ? value(a.pre_gamma, 0.f) : 0.f;
    vf[256 * W + at] =
        i < a.cols ? a.mask.scale * value(a.gate_rows ? nullptr : a.gate, 1.f) * value(a.post_gamma, 1.f) : 0.f;
  }
  const ulonglong2* vectors = reinterpret_cast<const ulonglong2*>(smem) + w * 64 + lane;
  auto vector = [&](int v, Pairs& out) {
    const ulonglong2 lo = vectors[v * 64 * W], hi = vectors[v * 64 * W + 32];
    out[0] = lo.x; out[1] = lo.y; out[2] = hi.x; out[3] = hi.y;
  };
#pragma unroll
  for (int i = 0; i < 2 * kSums; ++i) own_sums[i * blockDim.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto sum_at = [&](int i, Pairs& v) {
    const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(own_sums + 2 * i * blockDim.x),
                     hi = *reinterpret_cast<const ulonglong2*>(own_sums + (2 * i + 1) * blockDim.x);
    v[0] = lo.x; v[1] = lo.y; v[2] = hi.x; v[3] = hi.y;
  };
  auto put_sum = [&](int i, const Pairs& v) {
    *reinterpret_cast<ulonglong2*>(own_sums + 2 * i * blockDim.x) = make_ulonglong2(v[0], v[1]);
    *reinterpret_cast<ulonglong2*>(own_sums + (2 * i + 1) * blockDim.x) = make_ulonglong2(v[2], v[3]);
  };
  const float inv_n = 1.f / (float)a.cols;
  const uint32_t per_row = (uint32_t)a.cols / 8;
  int flip = 0, stage = 0;
  const uint8_t* from = ring;
  uint32_t parity = 0;
  __syncthreads();
  for (int row = first; row < a.rows; row += step) {
    Raw8<T> gate;  // (its row by the threads: in the ring it would take a group's room at 2560 columns)
    if (a.gate_rows) gate.load(static_cast<const T*>(a.gate) + (size_t)row * (uint32_t)a.cols + (active ? c : 0), 8);
    if (alive && !mbar_wait_warp(bars + stage, parity)) {
      alive = false;  // (the copy never came: nothing of this call is right, and nothing more is copied)
      latch_error(a.err, ERRBIT_TIMEOUT);
    }
    float4 st = pre || post ? *reinterpret_cast<const float4*>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (!pre) st.w = 0.f;  // (no norm's columns may hold anything)
    const uint8_t* values = from + 16;
    auto row_f = [&](int i, Pairs& v) { ld8_shared(reinterpret_cast<const float*>(values + i * f_bytes) + w * 256, lane, v); };
    auto row_t = [&](int i, Pairs& v) {
      ld8_shared(reinterpret_cast<const T*>(values + 2 * f_bytes + i * t_bytes) + w * 256, lane, v);
    };
    Pairs xh, e, yh, kept, p;
    float s[8];
    // all bits or none, per element: a dropped place is 0 whatever it holds
    fill(kept, __uint_as_float(~0u));
    keep(drop_words(a.mask, ps, &keys, (unsigned long long)(uint32_t)row * per_row + (uint32_t)c / 8), ps, kept);
    row_f(0, e);
    row_t(0, yh);
    if (partly && !active) {
      fill(e, 0.f);
      fill(yh, 0.f);
      fill(kept, 0.f);
    }
    uint64_t s2[8];
    if (pre) {
      Pairs dh;
      row_f(1, xh);
      row_t(1, dh);
      if (partly && !active) {
        fill(xh, st.z);
        fill(dh, 0.f);
      }
      Pairs sx, sd;
      sum_at(0, sx);
      sum_at(1, sd);
      vector(0, p);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xh[k] = f2_mul(f2_add(xh[k], f2_both(-st.z)), f2_both(st.w));
        sx[k] = f2_fma(dh[k], xh[k], sx[k]);
        sd[k] = f2_add(dh[k], sd[k]);
        const uint64_t gg = f2_mul(dh[k], p[k]);
        if (!RMS) s2[0] = k ? f2_add(s2[0], gg) : gg;
        s2[1] = k ? f2_fma(gg, xh[k], s2[1]) : f2_mul(gg, xh[k]);
        e[k] = f2_fma(f2_both(st.w), gg, e[k]);
      }
      put_sum(0, sx);
      put_sum(1, sd);
    } else {
      fill(xh, 0.f);
      s2[0] = s2[1] = 0;
    }
    if (post) {
      Pairs cg;
      vector(1, cg);
      if (a.gate_rows) {
        gate.get(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) cg[k] = f2_mul(cg[k], p[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t ck = cg[k] & kept[k];
        yh[k] = f2_mul(f2_add(yh[k], f2_both(-st.x)), f2_both(st.y));
        const uint64_t ce = f2_mul(ck, e[k] & kept[k]), cyh = f2_mul(ck, yh[k]);
        if (!RMS) {
          s2[2] = k ? f2_add(s2[2], ce) : ce;
          s2[3] = k ? f2_add(s2[3], ck) : ck;
          s2[4] = k ? f2_fma(ck, xh[k], s2[4]) : f2_mul(ck, xh[k]);
          s2[6] = k ? f2_add(s2[6], cyh) : cyh;
        }
        s2[5] = k ? f2_fma(ce, yh[k], s2[5]) : f2_mul(ce, yh[k]);
        s2[7] = k ? f2_fma(cyh, xh[k], s2[7]) : f2_mul(cyh, xh[k]);
      }
    } else {
      s2[2] = s2[3] = s2[4] = s2[5] = s2[6] = s2[7] = 0;
    }
    // the row's sums over the group's warps: value i of a warp stands with its lanes `per` i and on
    constexpr int kRowSums = RMS ? 4 : 8, per = 32 / kRowSums;
    float total;
    if constexpr (RMS) {
      float v[4] = {f2_sum(s2[1]), f2_sum(s2[5]), f2_sum(s2[7]), 0.f};
      total = warp_sum4(v, lane);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = f2_sum(s2[i]);
      total = warp_sum8(s, lane);
    }
    if (W > 1) {
      if (lane % per == 0) red[flip][warp][lane / per] = total;
      named_bar_sync(1 + group, 32 * W);
      total = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i += per)
        if (i + lane % per < W) total += red[flip][group * W + i + lane % per][lane / per];
#pragma unroll
      for (int o = per / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      flip ^= 1;
    } else {
      __syncwarp();
    }
    // the whole group has this row in its registers: the stage takes the next one
    if (w == 0 && lane == 0) arrive(row + kStages * step, stage);
    float A = 0.f, B, m0 = 0.f, m1;
    if constexpr (RMS) {
      B = st.w * __shfl_sync(0xffffffffu, total, 0) * inv_n;
      m1 = (__shfl_sync(0xffffffffu, total, per) - B * __shfl_sync(0xffffffffu, total, 2 * per)) * inv_n;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = __shfl_sync(0xffffffffu, total, per * i);
      A = st.w * s[0] * inv_n;
      B = st.w * s[1] * inv_n;
      m0 = (s[2] - A * s[3] - B * s[4]) * inv_n;
      m1 = (s[5] - A * s[6] - B * s[7]) * inv_n;
    }
    Pairs q, out;
    const size_t at = (size_t)row * (uint32_t)a.cols + c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      e[k] = f2_fma(f2_both(-B), xh[k], RMS ? e[k] : f2_add(e[k], f2_both(-A)));  // now G
      out[k] = f2_mul(f2_both(a.residual_scale), e[k]);
      q[k] = e[k] & kept[k];  // (the dropout's scale comes with p)
    }
    if (active) st8(a.dx + at, out);
    vector(1, p);
    if (!post) {
#pragma unroll
      for (int k = 0; k < 4; ++k) yh[k] &= kept[k];  // (y as it came)
    }
    if (a.gate_rows) {
      Pairs n, own_gate, beta;
      gate.get(own_gate);
      fill(beta, 0.f);
      if (a.post_beta && active) ld8(static_cast<const T*>(a.post_beta) + c, beta);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        n[k] = f2_mul(q[k], f2_fma(yh[k], p[k], f2_mul(f2_both(a.mask.scale), beta[k])));
        q[k] = f2_mul(q[k], own_gate[k]);
      }
      if (a.d_gate && active) st8(static_cast<T*>(a.d_gate) + at, n);
    }
    Pairs sp, sq;
    sum_at(2, sp);
    sum_at(3, sq);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      sp[k] = f2_fma(q[k], yh[k], sp[k]);
      sq[k] = f2_add(q[k], sq[k]);
      out[k] = f2_mul(p[k], q[k]);
      if (post) out[k] = f2_mul(f2_both(st.y), f2_fma(f2_both(-m1), yh[k], RMS ? out[k] : f2_add(out[k], f2_both(-m0))));
    }
    put_sum(2, sp);
    put_sum(3, sq);
    if (active) st8(static_cast<T*>(a.dy) + at, out);
    from += stage_bytes;
    if (++stage == kStages) {
      stage = 0;
      from = ring;
      parity ^= 1;
    }
  }
  if (!alive) {  // copies still on their way get as long again, whichever phase they belong to
    for (int i = 0; i < 2 * kStages; ++i) mbar_wait_warp(bars + i / 2, i & 1);
  }
  // the groups' sums are added in order
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem + 2048 * W);
  for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
    const int place = (((col >> 2 & 1) * blockDim.x) + (col >> 8) * 32 + (col >> 3 & 31)) * 4 + (col & 3);
#pragma unroll
    for (int s = 0; s < kSums; ++s) {
      float v = 0.f;
      for (int g = 0; g < groups; ++g) v += all[place + (2 * s * blockDim.x + g * W * 32) * 4];
      partial[((size_t)blockIdx.x * kSums + s) * a.cols + col] = s < 2 ? v : v * a.mask.scale;
    }
  }
}

// Any alignment, and rows of up to 8192 columns: the same sums, rows read where they are used (the next one is
// brought into the L2) and parameters from the L1; a lane owns 8 G columns, G = 2 with its column sums in shared
// memory.  One row a block at a time, then: 4096 x 5120 180 us, 2560 x 8192 150, 16384 x 1283 243, all far from the
// memory's time (56.5): a row's loads, sums and second reads of its parameters follow one another with nothing of the
// next row in shared memory, and 128 registers spill 72 to 136 bytes.
template <typename T, bool VEC, int G>
__global__ void __launch_bounds__(512, 1)
    block_norm_bwd_any_kernel(const BlockNormArgs a, int W, int groups, float* __restrict__ partial) {
  extern __shared__ __align__(16) float sums[];  // [kSums][cols], or each lane's own
  __shared__ float red[2][kBwdWarps][8];  // the two latest rows' sums of every warp
  grid_dependency_launch();
  __shared__ PhiloxKeys keys;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / W, w = warp - group * W;
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr;
  const long long first = (long long)blockIdx.x * groups + group, step = (long long)gridDim.x * groups;
  const PhiloxState ps = philox_state(a.mask);
  philox_keys(ps, &keys);
  const int own_left = a.cols - w * 256 * G;
  auto load = [&](const void* p, size_t at, int left, Pairs& out) {
    span_load<VEC>(static_cast<const T*>(p) + at, left, lane, out);
  };
  // G = 2: sum i of a lane's eight columns of its span g, in two halves
  auto own_sums = [&](int i, int g) { return reinterpret_cast<ulonglong2*>(sums) + ((i * G + g) * W + w) * 64 + lane; };
  Pairs acc[G == 1 ? kSums : 1];
#pragma unroll
  for (int i = 0; i < (G == 1 ? kSums : 1); ++i) fill(acc[i], 0.f);
  if constexpr (G > 1) {
    for (int i = threadIdx.x; i < kSums * G * W * 256; i += blockDim.x) sums[i] = 0.f;
  }
  __syncthreads();
  const float inv_n = 1.f / (float)a.cols;
  const uint32_t per_row = (uint32_t)(a.cols + 7) / 8;
  const uint64_t scale = f2_both(a.mask.scale), alpha = f2_both(a.residual_scale);
  int flip = 0;
  auto statistics = [&](long long row) {
    return (pre || post) && row < a.rows ? __ldg(reinterpret_cast<const float4*>(a.stats) + row)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 next = statistics(first);
  for (long long row = first; row < a.rows; row += step) {
    const float4 st = next;
    next = statistics(row + step);
    // the next row into the L2
    if (VEC && w == 0 && lane == 0 && row + step < a.rows) {
      const size_t at = (size_t)(row + step) * a.cols;
      const uint32_t t_bytes = (uint32_t)a.cols * sizeof(T);
      if (a.d_x_out) bulk_prefetch(a.d_x_out + at, 4 * (uint32_t)a.cols);
      if (pre) bulk_prefetch(a.x_out + at, 4 * (uint32_t)a.cols);
      bulk_prefetch(static_cast<const T*>(a.y) + at, t_bytes);
      if (pre) bulk_prefetch(static_cast<const T*>(a.d_h) + at, t_bytes);
      if (a.gate_rows) bulk_prefetch(static_cast<const T*>(a.gate) + at, t_bytes);
    }
    if (!VEC && row + step < a.rows) {
      const size_t at = (size_t)(row + step) * a.cols + w * 256 * G;
      constexpr int kLine = 128 / sizeof(T);
      if (32 * lane < min(256 * G, own_left)) {
        if (a.d_x_out) prefetch_l2(a.d_x_out + at + 32 * lane);
        if (pre) prefetch_l2(a.x_out + at + 32 * lane);
      }
      if (kLine * lane < min(256 * G, own_left)) {
        prefetch_l2(static_cast<const T*>(a.y) + at + kLine * lane);
        if (pre) prefetch_l2(static_cast<const T*>(a.d_h) + at + kLine * lane);
        if (a.gate_rows) prefetch_l2(static_cast<const T*>(a.gate) + at + kLine * lane);
      }
    }
    const uint64_t minus_x = f2_both(-st.z), rx = f2_both(st.w), minus_y = f2_both(-st.x), ry = f2_both(st.y);
    Pairs xh[G], e[G], yh[G];
    uint4 words[G];
    uint64_t s2[8] = {};
    auto add = [&](int g, int i, const Pairs& v) {  // (products are added as they are made)
      if constexpr (G == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = f2_add(acc[i][k], v[k]);
      } else {
        ulonglong2* to = own_sums(i, g);
        ulonglong2 lo = to[0], hi = to[32];
        lo.x = f2_add(lo.x, v[0]); lo.y = f2_add(lo.y, v[1]);
        hi.x = f2_add(hi.x, v[2]); hi.y = f2_add(hi.y, v[3]);
        to[0] = lo;
        to[32] = hi;
      }
    };
    auto add_product = [&](int g, int i, const Pairs& v, const Pairs& by) {
      if constexpr (G == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = f2_fma(v[k], by[k], acc[i][k]);
      } else {
        Pairs p;
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = f2_mul(v[k], by[k]);
        add(g, i, p);
      }
    };
    // c before the mask (made again after the exchange: registers are short)
    auto factors = [&](int g, size_t base, Pairs& c) {
      Pairs p;
      const int c0 = (g * W + w) * 256, left = a.cols - c0;
      load(a.post_gamma, c0, left, c);
      if (a.gate) {
        load(a.gate, a.gate_rows ? base : c0, left, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = f2_mul(c[k], p[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = f2_mul(c[k], scale);
    };
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (g * W + w) * 256, left = a.cols - c0;
      const size_t base = (size_t)row * a.cols + c0;
      Pairs dh, p;
      fill(e[g], 0.f);
      if (a.d_x_out) span_load<VEC>(a.d_x_out + base, left, lane, e[g]);
      load(a.y, base, left, yh[g]);
      if (pre) {
        span_load<VEC>(static_cast<const float*>(a.x_out) + base, left, lane, xh[g]);
        load(a.d_h, base, left, dh);
      }
      words[g] = span_words<VEC>(
          a.mask, drop_words(a.mask, ps, &keys, (unsigned long long)row * per_row + c0 / 8 + lane), lane);
      if (pre) {
        load(a.pre_gamma, c0, left, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) xh[g][k] = f2_mul(f2_add(xh[g][k], minus_x), rx);
        span_trim<VEC>(left, lane, xh[g]);
        add_product(g, 0, dh, xh[g]);
        add(g, 1, dh);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t gg = f2_mul(dh[k], p[k]);
          s2[0] = f2_add(s2[0], gg);
          s2[1] = f2_fma(gg, xh[g][k], s2[1]);
          e[g][k] = f2_fma(rx, gg, e[g][k]);
        }
      } else {
        fill(xh[g], 0.f);
      }
      if (post) {
        Pairs c, ek;  // (0 where they are dropped, whatever d_x_out holds there)
        factors(g, base, c);
        keep(words[g], ps, c);
#pragma unroll
        for (int k = 0; k < 4; ++k) ek[k] = e[g][k];
        keep(words[g], ps, ek);
#pragma unroll
        for (int k = 0; k < 4; ++k) yh[g][k] = f2_mul(f2_add(yh[g][k], minus_y), ry);
        span_trim<VEC>(left, lane, yh[g]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t ce = f2_mul(c[k], ek[k]), cyh = f2_mul(c[k], yh[g][k]);
          s2[2] = f2_add(s2[2], ce);
          s2[3] = f2_add(s2[3], c[k]);
          s2[4] = f2_fma(c[k], xh[g][k], s2[4]);
          s2[5] = f2_fma(ce, yh[g][k], s2[5]);
          s2[6] = f2_add(s2[6], cyh);
          s2[7] = f2_fma(cyh, xh[g][k], s2[7]);
        }
      }
    }
    float s[8];
    if (pre || post) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = f2_sum(s2[i]);
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
    const float A = pre && !a.rms ? st.w * s[0] * inv_n : 0.f, B = pre ? st.w * s[1] * inv_n : 0.f;
    const float m0 = post && !a.rms ? (s[2] - A * s[3] - B * s[4]) * inv_n : 0.f;
    const float m1 = post ? (s[5] - A * s[6] - B * s[7]) * inv_n : 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (g * W + w) * 256, left = a.cols - c0;
      const size_t base = (size_t)row * a.cols + c0;
      Pairs out, q;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e[g][k] = f2_fma(f2_both(-B), xh[g][k], f2_add(e[g][k], f2_both(-A)));  // now G
        out[k] = f2_mul(alpha, e[g][k]);
        q[k] = f2_mul(scale, e[g][k]);
      }
      span_store<VEC>(a.dx + base, left, lane, out);
      keep(words[g], ps, q);
      if (a.gate_rows) {
        Pairs gate, n;
        load(a.gate, base, left, gate);
#pragma unroll
        for (int k = 0; k < 4; ++k) n[k] = yh[g][k];
        if (post) {
          Pairs p, b;
          load(a.post_gamma, c0, left, p);
          fill(b, 0.f);
          if (a.post_beta) load(a.post_beta, c0, left, b);
#pragma unroll
          for (int k = 0; k < 4; ++k) n[k] = f2_fma(n[k], p[k], b[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          n[k] = f2_mul(n[k], q[k]);
          q[k] = f2_mul(q[k], gate[k]);
        }
        keep(words[g], ps, n);
        if (a.d_gate) span_store<VEC>(static_cast<T*>(a.d_gate) + base, left, lane, n);
      }
      if (!post) {
        // (a dropped value adds nothing, whatever y holds there)
        keep(words[g], ps, yh[g]);
      }
      add_product(g, 2, q, yh[g]);
      add(g, 3, q);
      if (post) {
        Pairs c;
        factors(g, base, c);
        keep(words[g], ps, c);
        keep(words[g], ps, e[g]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          out[k] = f2_mul(ry, f2_fma(f2_both(-m1), yh[g][k], f2_fma(c[k], e[g][k], f2_both(-m0))));
      } else {
        if (a.gate && !a.gate_rows) {
          load(a.gate, c0, left, out);
#pragma unroll
          for (int k = 0; k < 4; ++k) out[k] = f2_mul(out[k], q[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) out[k] = q[k];
        }
      }
      span_store<VEC>(static_cast<T*>(a.dy) + base, left, lane, out);
    }
  }
  if constexpr (G == 1) {
    // the groups add their sums in order
    const int c0 = w * 256;
    for (int turn = 0; turn < groups; ++turn) {
      if (turn == group) {
#pragma unroll
        for (int i = 0; i < kSums; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int col = span_col<VEC>(lane, k);
            if (col < own_left) {
              const float v = k & 1 ? f2_hi(acc[i][k / 2]) : f2_lo(acc[i][k / 2]);
              float* to = sums + (size_t)i * a.cols + c0 + col;
              *to = turn ? *to + v : v;
            }
          }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < kSums * a.cols; i += blockDim.x)
      partial[(size_t)blockIdx.x * kSums * a.cols + i] = sums[i];
  } else {
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int c0 = (g * W + w) * 256;
        const ulonglong2 lo = own_sums(i, g)[0], hi = own_sums(i, g)[32];
        const Pairs v = {lo.x, lo.y, hi.x, hi.y};
        span_store<VEC>(partial + ((size_t)blockIdx.x * kSums + i) * a.cols + c0, a.cols - c0, lane, v);
      }
  }
}

// The parameters' gradients from the blocks' column sums, in a fixed order: warp w of a block adds blocks
// w, w + 32, ... of 32 columns, then the warps' sums are added in order.  Even blocks: the sums of pre, odd: of post.
template <typename T>
__global__ void __launch_bounds__(1024) block_norm_sums_kernel(const BlockNormArgs a, const float* __restrict__ partial,
                                                              int blocks) {
  __shared__ float part[2][32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, post = blockIdx.x & 1, c = (blockIdx.x >> 1) * 32 + lane;
  grid_dependency_wait();
  float s0 = 0.f, s1 = 0.f;
  if (c < a.cols) {
#pragma unroll 5
    for (int b = warp; b < blocks; b += 32) {
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
  for (int i = 1; i < 32; ++i) {
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
  s.groups = s.G == 2 ? 1 : std::min(kMaxGroups, kBwdWarps / s.W);
  s.blocks = std::max(1, std::min(num_sms, (rows + s.groups - 1) / s.groups));
  return s;
}

constexpr size_t kSmemMax = 227 * 1024 - 2048;  // (the rest: static shared memory)

// Lets a kernel have `smem` bytes of dynamic shared memory.  The limit belongs to the kernel, for all host threads: it
// is always set to `most`, what any shape may need, so that no call lowers it under another's launch.
template <typename Kernel>
cudaError_t allow_smem(Kernel k, size_t smem, size_t most) {
  return smem <= 40 * 1024 ? cudaSuccess : cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

template <typename T, bool VEC, int G>
cudaError_t launch_bwd_any(const BlockNormArgs& a, const BwdShape& s, float* partial, cudaStream_t st) {
  const size_t smem = sizeof(float) * kSums * (G == 1 ? a.cols : G * s.W * 256);
  constexpr size_t kMost = sizeof(float) * kSums * (G == 1 ? 16 * 256 : ESM_BLOCK_NORM_MAX_COLS);
  const cudaError_t e = allow_smem(block_norm_bwd_any_kernel<T, VEC, G>, smem, kMost);
  if (e != cudaSuccess) return e;
  block_norm_bwd_any_kernel<T, VEC, G><<<s.blocks, 32 * s.W * s.groups, smem, st>>>(a, s.W, s.groups, partial);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const BlockNormArgs& a, bool vec, float* partial, int num_sms, cudaStream_t st) {
  BwdShape s = bwd_shape(a.rows, a.cols, num_sms);
  // a group's rows and sums, behind the vectors (1 KB more: lanes past a row's end read on behind it)
  const size_t group = ((size_t)a.cols * (8 + 2 * sizeof(T)) + 16) * kStages + (size_t)1024 * kSums * s.W;
  const size_t fixed = 2048 * s.W + 1024, fits = (kSmemMax - fixed) / group;
  cudaError_t e;
  if (s.G == 2) {
    e = vec ? launch_bwd_any<T, true, 2>(a, s, partial, st) : launch_bwd_any<T, false, 2>(a, s, partial, st);
  } else if (!vec || fits == 0) {
    s.groups = std::min(s.groups, 16 / s.W);
    e = vec ? launch_bwd_any<T, true, 1>(a, s, partial, st) : launch_bwd_any<T, false, 1>(a, s, partial, st);
  } else {
    s.groups = (int)std::min({(size_t)s.groups, fits, (size_t)(kWarpsOf<T> / s.W)});
    const size_t smem = fixed + group * s.groups;
    const auto kernel = a.rms ? block_norm_bwd_kernel<T, true> : block_norm_bwd_kernel<T, false>;
    e = allow_smem(kernel, smem, kSmemMax);
    if (e != cudaSuccess) return e;
    kernel<<<s.blocks, 32 * s.W * s.groups, smem, st>>>(a, s.W, s.groups, partial);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_after(block_norm_sums_kernel<T>, 2 * ((a.cols + 31) / 32), 1024, st, a, (const float*)partial, s.blocks);
}

// W warps to a row of up to 4096 columns.  Registers for 800 threads an SM with bfloat16 blocks (72 each; 16384 x
// 1280: 46.3 us, for 640 threads 53.9, for 960 48.7) and for 640 with float32 ones (55.7 us, for 512 64.2).
template <typename T, int W>
void launch_fwd_as(const BlockNormArgs& a, const RowShape& s, int spans, int num_sms, cudaStream_t st) {
  constexpr int kThreads = 32 * W, kBlocks = std::min(24, (sizeof(T) == 2 ? 800 : 640) / kThreads);
  if (spans > 8)
    block_norm_kernel<T, true, W, 1, 2, kThreads, kBlocks><<<(unsigned)a.rows, kThreads, 0, st>>>(a, s);
  else if (a.rows > 2 * num_sms)
    block_norm_kernel<T, true, W, 2, 1, kThreads, kBlocks><<<(unsigned)((a.rows + 1) / 2), kThreads, 0, st>>>(a, s);
  else
    block_norm_kernel<T, true, W, 1, 1, kThreads, 1><<<(unsigned)a.rows, kThreads, 0, st>>>(a, s);
}

template <typename T>
cudaError_t launch_fwd(const BlockNormArgs& a, bool vec, int num_sms, cudaStream_t st) {
  const int spans = (a.cols + 255) / 256;
  const bool by_width = vec && spans <= 16;
  const int G = vec && spans > 8 ? 2 : 1, W = (spans + G - 1) / G;
  RowShape s;
  s.inv_cols = 1.f / (float)a.cols;
  s.last = (float)(a.cols - 256 * G * (W - 1));
  s.inv_last = 1.f / s.last;
  if (!by_width) {
    const unsigned rows = (unsigned)a.rows;
    if (vec) {
      // (4096 x 5120: 58 us, 2560 x 8192: 64; a span a warp, one block an SM: 102 and 100.  64 registers spill 112 bytes,
      // 392 with float32 blocks, which take 88 and 96)
      block_norm_kernel<T, true, 0, 1, 2, 512, 2><<<rows, 32 * W, 0, st>>>(a, s);
    } else if (spans <= 8) {
      block_norm_kernel<T, false, 0, 1, 1, 256, 4><<<rows, 32 * W, 0, st>>>(a, s);
    } else {
      block_norm_kernel<T, false, 0, 1, 1, 1024, 1><<<rows, 32 * W, 0, st>>>(a, s);
    }
    return cudaGetLastError();
  }
  switch (W) {
    case 1: launch_fwd_as<T, 1>(a, s, spans, num_sms, st); break;
    case 2: launch_fwd_as<T, 2>(a, s, spans, num_sms, st); break;
    case 3: launch_fwd_as<T, 3>(a, s, spans, num_sms, st); break;
    case 4: launch_fwd_as<T, 4>(a, s, spans, num_sms, st); break;
    case 5: launch_fwd_as<T, 5>(a, s, spans, num_sms, st); break;
    case 6: launch_fwd_as<T, 6>(a, s, spans, num_sms, st); break;
    case 7: launch_fwd_as<T, 7>(a, s, spans, num_sms, st); break;
    default: launch_fwd_as<T, 8>(a, s, spans, num_sms, st); break;
  }
  return cudaGetLastError();
}

// A row's or parameter's eight values at a time (cols % 8 == 0 is part of it).
bool all_on_eights(const BlockNormArgs& a, bool bf16) {
  const int es = bf16 ? 2 : 4;
  for (const void* p : {a.y, (const void*)a.h, a.d_h, (const void*)a.dy, a.post_gamma, a.post_beta, a.pre_gamma, a.pre_beta,
                        a.gate, a.gate_rows ? (const void*)a.d_gate : nullptr})
    if (!rows_on_eights(p, a.cols, es)) return false;
  for (const float* p : {a.x, (const float*)a.x_out, a.d_x_out, (const float*)a.dx})
    if (!rows_on_eights(p, a.cols, 4)) return false;
  return true;
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, bool bf16, int num_sms, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const bool vec = all_on_eights(a, bf16);
  return bf16 ? launch_fwd<__nv_bfloat16>(a, vec, num_sms, st) : launch_fwd<float>(a, vec, num_sms, st);
}

size_t block_norm_bwd_workspace_bytes(int rows, int cols, int num_sms) {
  return sizeof(float) * kSums * (size_t)cols * bwd_shape(rows, cols, num_sms).blocks;
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& a, bool bf16, void* workspace, int num_sms, cudaStream_t st) {
  const bool vec = all_on_eights(a, bf16);
  float* partial = static_cast<float*>(workspace);
  return bf16 ? launch_bwd<__nv_bfloat16>(a, vec, partial, num_sms, st) : launch_bwd<float>(a, vec, partial, num_sms, st);
}

}  // namespace esm
