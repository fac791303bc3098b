// Variable-length bidirectional attention over packed sequences, fp32 (the ESM_FP32
// precision of the small fp32 configuration; bf16 and FP8 encoders use the tcgen05 kernel
// in attention_tc.cu).
//
// Section 3.2 of the hotelren.com guide ("生物大模型训练加速实战") runs every layer over
// cu_seqlens (thd format); the BioNeMo ESM-2 model card describes a bidirectional
// (BERT-style) encoder.  So each token attends to every token of its own sequence and to
// nothing else:
//
//   o_t = sum_s softmax_s(q_t . k_s / sqrt(dh)) v_s,   s over the sequence of t,
//
// or, with a window (attention_window_f32_kernel), over the keys s <= t + right with s >= t - left or
// s < sinks (positions in the sequence); a row that sees no key is zero, one whose visible scores are
// all -inf is NaN.
#include "common.cuh"
#include "internal.h"

namespace esm {
namespace {

// Output row t of head h by one warp: lanes split the keys, each keeps a running max / sum / output,
// merged across lanes at the end.
__device__ __forceinline__ void attention_f32_row(const float* __restrict__ qkv, float* __restrict__ o, int d, int heads,
                                                  const PackBuffers& pb, const AttnWindow& win, int t, int h) {
  const int lane = threadIdx.x & 31;
  const int dh = d / heads;
  const int seg = pb.seg_id[t];
  const int start = pb.seg_start[seg];
  const int klen = pb.seg_klen[seg];
  const int ld = 3 * d;
  float q[64];
#pragma unroll
  for (int c = 0; c < 64; ++c) q[c] = c < dh ? qkv[(size_t)t * ld + h * dh + c] : 0.f;
  const float scale = 1.f / sqrtf((float)dh);
  float m = -INFINITY, l = 0.f, acc[64];
#pragma unroll
  for (int c = 0; c < 64; ++c) acc[c] = 0.f;
  // the visible keys: [0, ns) and [lo, end)
  const int pos = t - start;
  const int end = win.right < 0 ? klen : min(klen, pos + win.right + 1);
  const int lo = win.left < 0 ? 0 : max(0, pos - win.left), ns = min(win.sinks, min(lo, end));
  const int n = ns + max(0, end - lo);
  for (int i = lane; i < n; i += 32) {
    const int j = i < ns ? i : lo + i - ns;
    const float* kr = qkv + (size_t)(start + j) * ld + d + h * dh;
    const float* vr = qkv + (size_t)(start + j) * ld + 2 * d + h * dh;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 64; ++c)
      if (c < dh) s = fmaf(q[c], kr[c], s);
    s *= scale;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float corr = expf(m - base), p = expf(s - base);
    l = l * corr + p;
#pragma unroll
    for (int c = 0; c < 64; ++c)
      if (c < dh) acc[c] = acc[c] * corr + p * vr[c];
    m = mn;
  }
  float M = m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float f = (m == -INFINITY) ? 0.f : expf(m - M);
  l *= f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
  for (int c = 0; c < 64; ++c) {
    if (c >= dh) break;
    float v = acc[c] * f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0) o[(size_t)t * d + h * dh + c] = n > 0 ? v / l : 0.f;
  }
}

// fp32 attention (the ESM_FP32 precision): one warp per (query row, head).
__global__ void attention_f32_kernel(const float* __restrict__ qkv, float* __restrict__ o, int d, int heads, int T,
                                     PackBuffers pb) {
  const int gw = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (gw >= T * heads) return;
  attention_f32_row(qkv, o, d, heads, pb, AttnWindow{-1, -1, 0}, gw / heads, gw - (gw / heads) * heads);
}

// (out of line: its 64 accumulators per lane are not the windowed kernel's)
__device__ __noinline__ void attention_f32_row_again(const float* qkv, float* o, int d, int heads, const PackBuffers& pb,
                                                     const AttnWindow& win, int t, int h) {
  attention_f32_row(qkv, o, d, heads, pb, win, t, h);
}

// The windowed form: a block per 32 consecutive rows of the batch (of one sequence or several) and
// head, with a running maximum and sum per row over tiles of 64 keys.  The keys of a block are the
// sinks of its first row's sequence, then the packed rows from the first to the last that any of its
// rows sees in its band (a later sequence begins inside the block, and so within those rows).
// Thread (ty, tx) holds rows 4 ty .. + 3 and columns 4 tx .. + 3 of the scores and of O.  A zero weight
// times an infinite or NaN value is NaN: a row that ends up not finite, but for its own scores, is
// done again over its visible keys alone.
//
// 16 products per two 16-byte loads of shared memory, four barriers per tile and no loads ahead of it:
// one sequence of 1024 tokens, 8 heads, window 1024 + 1024, takes 143 us a call after an L2 flush, five
// times its products at the FMA rate (the full attention's warp per row: 3700).
constexpr int FQ = 32, FK = 64, FD = 64;
__global__ void __launch_bounds__(128) attention_window_f32_kernel(const float* __restrict__ qkv, float* __restrict__ o,
                                                                   int d, int heads, int T, PackBuffers pb,
                                                                   AttnWindow win) {
  __shared__ __align__(16) float s_q[FD][FQ + 4];       // [column][row]
  __shared__ __align__(16) float s_kp[FD * (FK + 4)];   // K as [column][key], then P as [key][row]
  __shared__ __align__(16) float s_v[FK][FD + 4];       // [key][column]
  __shared__ int s_start[FQ], s_ns[FQ], s_lo[FQ], s_end[FQ];  // first packed row, sinks, band (packed rows)
  __shared__ int s_range[2], s_sinks;
  __shared__ unsigned s_redo;
  const int t0 = blockIdx.x * FQ, h = blockIdx.y, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int dh = d / heads, ld = 3 * d;
  if (tid < FQ) {
    const int t = t0 + tid;
    int start = 0, ns = 0, lo = 0, end = 0;
    if (t < T) {
      const int seg = pb.seg_id[t], klen = pb.seg_klen[seg];
      start = pb.seg_start[seg];
      const int pos = t - start;
      end = win.right < 0 ? klen : min(klen, pos + win.right + 1);
      lo = win.left < 0 ? 0 : max(0, pos - win.left);
      ns = max(0, min(win.sinks, min(lo, end)));
      lo += start;
      end += start;
    }
    s_start[tid] = start;
    s_ns[tid] = ns;
    s_lo[tid] = lo;
    s_end[tid] = end;
    const bool some = end > lo;
    const int first = __reduce_min_sync(0xffffffffu, some ? lo : 0x7fffffff);
    const int last = __reduce_max_sync(0xffffffffu, some ? end : 0);
    const int start0 = __shfl_sync(0xffffffffu, start, 0);
    const int most = __reduce_max_sync(0xffffffffu, start == start0 ? ns : 0);
    if (tid == 0) {
      s_range[0] = first < last ? first : 0;
      s_range[1] = first < last ? last : 0;
      s_sinks = first < last ? max(0, min(most, first - start0)) : most;
      s_redo = 0u;
    }
  }
  for (int i = tid; i < FQ * FD; i += 128) {
    const int row = i & (FQ - 1), c = i / FQ;
    s_q[c][row] = t0 + row < T && c < dh ? qkv[(size_t)(t0 + row) * ld + h * dh + c] : 0.f;
  }
  __syncthreads();
  const int start0 = s_start[0], nsink = s_sinks, first = s_range[0];
  const int n_keys = nsink + s_range[1] - first;
  const float scale = 1.f / sqrtf((float)dh);
  float m[4], l[4], acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  }
  for (int k0 = 0; k0 < n_keys; k0 += FK) {
    auto packed_row = [&](int k) { return k < nsink ? start0 + k : first + k - nsink; };
    __syncthreads();  // the previous tile's P and V have been read
    for (int i = tid; i < FK * FD / 4; i += 128) {
      const int key = i & (FK - 1), c = i / FK * 4, k = k0 + key;
      float kv[4] = {0.f, 0.f, 0.f, 0.f}, vv[4] = {0.f, 0.f, 0.f, 0.f};
      if (k < n_keys) {
        const float* src = qkv + (size_t)packed_row(k) * ld + d + h * dh + c;
        if (dh == FD) {  // (then rows and heads start on 16 bytes)
          *reinterpret_cast<float4*>(kv) = *reinterpret_cast<const float4*>(src);
          *reinterpret_cast<float4*>(vv) = *reinterpret_cast<const float4*>(src + d);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < dh) {
              kv[j] = src[j];
              vv[j] = src[d + j];
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s_kp[(c + j) * (FK + 4) + key] = kv[j];
      *reinterpret_cast<float4*>(&s_v[key][c]) = *reinterpret_cast<float4*>(vv);
    }
    __syncthreads();
    float s[4][4] = {};
#pragma unroll 8
    for (int c = 0; c < FD; ++c) {
      float a[4], b[4];
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(&s_q[c][4 * ty]);
      *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(&s_kp[c * (FK + 4) + 4 * tx]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a[i], b[j], s[i][j]);
    }
    __syncthreads();  // K has been read: P takes its place
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 4 * tx + j, g = packed_row(k);
        const bool seen = k < n_keys && ((g >= s_lo[row] && g < s_end[row]) ||
                                         (g >= s_start[row] && g < s_start[row] + s_ns[row]));
        s[i][j] = seen ? s[i][j] * scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
      const float corr = expf(m[i] - base);
      m[i] = mn;
      l[i] *= corr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = expf(s[i][j] - base);
        l[i] += s[i][j];
        acc[i][j] *= corr;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(&s_kp[(4 * tx + j) * (FQ + 4) + 4 * ty]) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < FK; ++k) {
      float a[4], b[4];
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(&s_kp[k * (FQ + 4) + 4 * ty]);
      *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(&s_v[k][4 * tx]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * ty + i, t = t0 + row;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
    // (a sum of 0: the row sees no key, or only scores of -inf; a NaN: a score of NaN or +inf)
    const bool sees = s_ns[row] > 0 || s_end[row] > s_lo[row], sums = l[i] > 0.f;
    const float inv = sums ? 1.f / l[i] : sees ? __int_as_float(0x7fffffff) : 0.f;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = sums ? acc[i][j] * inv : inv;
      odd |= sums && !(fabsf(v) <= 3.402823466e38f);
      if (t < T && 4 * tx + j < dh) o[(size_t)t * d + h * dh + 4 * tx + j] = v;
    }
    if (odd && t < T) atomicOr(&s_redo, 1u << row);
  }
  __syncthreads();
  // (rare) the rows set aside, a warp each
  int n = 0;
  for (unsigned todo = s_redo; todo != 0u; todo &= todo - 1, ++n)
    if ((n & 3) == (tid >> 5)) attention_f32_row_again(qkv, o, d, heads, pb, win, t0 + __ffs(todo) - 1, h);
}

}  // namespace

void launch_attention_f32(const float* qkv, float* o, int d, int heads, int T, const PackBuffers& pb,
                          cudaStream_t st) {
  if (T <= 0) return;
  const int warps = 4;
  const long long n = (long long)T * heads;
  attention_f32_kernel<<<(unsigned)((n + warps - 1) / warps), 32 * warps, 0, st>>>(qkv, o, d, heads, T, pb);
}

void launch_attention_window_f32(const float* qkv, float* o, int d, int heads, int T, const PackBuffers& pb,
                                 const AttnWindow& win, cudaStream_t st) {
  if (T <= 0) return;
  attention_window_f32_kernel<<<dim3((T + FQ - 1) / FQ, heads), 128, 0, st>>>(qkv, o, d, heads, T, pb, win);
}

}  // namespace esm
