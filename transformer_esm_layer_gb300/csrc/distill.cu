// Distillation from a teacher's top logits: the loss of a student's logits z [T, V] against K
// stored entries (id, logit) per token, and its gradient.
//
// With temperature t, q = softmax(z / t) over the vocabulary and p = softmax(l / t) over the
// row's usable teacher entries (0 <= id < V, logit l > -inf):
//
//   loss = t^2 sum_k p_k (log p_k - log q_{id_k}),  log q_v = z_v / t - lse,
//   lse  = log sum_v exp(z_v / t),
//   dloss/dz_v = t (q_v - sum_{k: id_k = v} p_k).
//
// A row without a usable entry is not scored: loss, lse and gradient 0, its logits unread.
// Logits are read once per call (forward: running maximum and sum per thread, merged in a
// fixed order; backward: q from the forward's lse, each value overwritten where it is read, so
// the gradient may take the logits' place).  Exponentials, sums and the loss are fp32 whatever
// the logits' type; the gradient is rounded once, to the logits' type.
//
// Both directions are bound by the logits' bytes.  Two forms: a warp per row with the row in
// registers up to kWarpVocab values, and a block per row above.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace esm {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWarpVocab = 256;      // a warp holds up to 8 values of the row per lane
constexpr int kWarpsPerBlock = 8;    // rows of a block, warp form
constexpr int kRowThreads = 256;     // threads of a row, block form; >= the entries of a row
static_assert(kDistillMaxK <= kRowThreads, "one teacher entry per thread");

template <typename E>
__device__ __forceinline__ float to_f(E v) {
  if constexpr (sizeof(E) == 2) return __bfloat162float(v);
  else return v;
}
template <typename E>
__device__ __forceinline__ E from_f(float v) {
  if constexpr (sizeof(E) == 2) return __float2bfloat16_rn(v);
  else return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The reference point of a running sum of exponentials: a maximum of -inf (nothing but -inf so
// far) is replaced by 0, which leaves every term 0.
__device__ __forceinline__ float anchor(float m) { return m == -INFINITY ? 0.f : m; }

// A teacher entry's id if it is usable, else -1; ids outside [-1, V) are reported.
__device__ __forceinline__ int usable_id(int id, float l, int V, unsigned* err) {
  if (id < -1 || id >= V) latch_error(err, ERRBIT_TOKEN);
  return id >= 0 && id < V && l != -INFINITY ? id : -1;
}

// Teacher softmax of one row by one warp, entries k = lane, lane + 32, ...: the maximum of l / t,
// and log and value of the sum.  n: usable entries.
struct Teacher {
  float m, sum;
  int n;
};
__device__ __forceinline__ Teacher teacher_stats(const int32_t* ids, const float* tl, int K, int V, float inv_t,
                                                 unsigned* err) {
  const int lane = threadIdx.x & 31;
  Teacher s{-INFINITY, 0.f, 0};
  for (int k = lane; k < K; k += 32) {
    if (usable_id(ids[k], tl[k], V, err) < 0) continue;
    s.m = fmaxf(s.m, tl[k] * inv_t);
    ++s.n;
  }
  s.m = anchor(warp_max(s.m));
  s.n = __reduce_add_sync(0xffffffffu, s.n);
  for (int k = lane; k < K; k += 32)
    if (usable_id(ids[k], tl[k], V, nullptr) >= 0) s.sum += expf(tl[k] * inv_t - s.m);
  s.sum = warp_sum(s.sum);
  return s;
}

// Loss of one row by one warp, from the row's lse.
template <typename E>
__device__ __forceinline__ float row_loss(const E* row, const int32_t* ids, const float* tl, int K, int V, float inv_t,
                                          float temperature, const Teacher& s, float lse) {
  const float log_sum = logf(s.sum), inv_sum = 1.f / s.sum;
  float acc = 0.f;
  for (int k = threadIdx.x & 31; k < K; k += 32) {
    const int id = usable_id(ids[k], tl[k], V, nullptr);
    if (id < 0) continue;
    const float a = tl[k] * inv_t - s.m;
    const float p = expf(a) * inv_sum;
    // an entry whose probability underflows adds nothing, whatever the student makes of it
    if (p != 0.f) acc = fmaf(p, (a - log_sum) - (to_f(row[id]) * inv_t - lse), acc);
  }
  return temperature * temperature * warp_sum(acc);
}

// ---------------------------------------------------------------- warp form
template <typename E, int N>
__global__ void __launch_bounds__(32 * kWarpsPerBlock)
    distill_warp_kernel(const E* __restrict__ logits, long long stride, const int32_t* __restrict__ ids,
                        const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                        float* __restrict__ token_loss, float* __restrict__ lse_out, float* __restrict__ part_loss,
                        int* __restrict__ part_count, unsigned* err) {
  __shared__ float s_loss[kWarpsPerBlock];
  __shared__ int s_count[kWarpsPerBlock];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float c = kLog2e * inv_t;
  float loss_acc = 0.f;
  int count = 0;
  for (int t = blockIdx.x * kWarpsPerBlock + warp; t < T; t += gridDim.x * kWarpsPerBlock) {
    const E* row = logits + (size_t)t * stride;
    const int32_t* id = ids + (size_t)t * K;
    const float* l = tl + (size_t)t * K;
    const Teacher s = teacher_stats(id, l, K, V, inv_t, err);
    float loss = 0.f, lse = 0.f;
    if (s.n > 0) {
      float z[N], m = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        z[i] = lane + 32 * i < V ? to_f(row[lane + 32 * i]) : -INFINITY;
        m = fmaxf(m, z[i]);
      }
      m = anchor(warp_max(m));
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) sum += ex2_approx((z[i] - m) * c);
      lse = fmaf(m, inv_t, logf(warp_sum(sum)));
      loss = row_loss(row, id, l, K, V, inv_t, temperature, s, lse);
      ++count;
    }
    if (lane == 0) {
      token_loss[t] = loss;
      if (lse_out) lse_out[t] = lse;
    }
    loss_acc += loss;
  }
  if (part_loss == nullptr) return;
  if (lane == 0) {
    s_loss[warp] = loss_acc;
    s_count[warp] = count;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float a = 0.f;
    int n = 0;
    for (int w = 0; w < kWarpsPerBlock; ++w) {
      a += s_loss[w];
      n += s_count[w];
    }
    part_loss[blockIdx.x] = a;
    part_count[blockIdx.x] = n;
  }
}

template <typename E, int N>
__global__ void __launch_bounds__(32 * kWarpsPerBlock)
    distill_bwd_warp_kernel(const E* logits, long long stride, const int32_t* __restrict__ ids,
                            const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                            const float* __restrict__ lse_in, const int* __restrict__ loss_count, E* d_logits,
                            long long d_stride, unsigned* err) {
  __shared__ float s_p[kWarpsPerBlock][32 * N];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = loss_count ? *loss_count : 1;
  const float amp = n > 0 ? temperature / (float)n : 0.f;
  float* p_row = s_p[warp];
  for (int t = blockIdx.x * kWarpsPerBlock + warp; t < T; t += gridDim.x * kWarpsPerBlock) {
    const E* row = logits + (size_t)t * stride;
    E* out = d_logits + (size_t)t * d_stride;
    const int32_t* id = ids + (size_t)t * K;
    const float* l = tl + (size_t)t * K;
    const Teacher s = teacher_stats(id, l, K, V, inv_t, err);
    if (s.n == 0 || amp == 0.f) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane + 32 * i < V) out[lane + 32 * i] = from_f<E>(0.f);
      continue;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) p_row[lane + 32 * i] = 0.f;
    __syncwarp();
    const float inv_sum = 1.f / s.sum;
    for (int k0 = 0; k0 < K; k0 += 32) {
      const int k = k0 + lane;
      const int v = k < K ? usable_id(id[k], l[k], V, nullptr) : -1;
      const float p = v >= 0 ? expf(l[k] * inv_t - s.m) * inv_sum : 0.f;
      const unsigned same = __match_any_sync(0xffffffffu, v);
      if (__any_sync(0xffffffffu, v >= 0 && (same & (same - 1)) != 0u)) {
        // an id stands there twice: one entry after the other
        for (int j = 0; j < 32; ++j) {
          if (lane == j && v >= 0) p_row[v] += p;
          __syncwarp();
        }
      } else if (v >= 0) {
        p_row[v] += p;
      }
      __syncwarp();
    }
    const float lse = lse_in[t];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = lane + 32 * i;
      if (v < V) {
        const float q = ex2_approx(fmaf(to_f(row[v]), inv_t, -lse) * kLog2e);
        out[v] = from_f<E>(amp * (q - p_row[v]));
      }
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- block form
// 16-byte unit of a row as floats.
template <typename E>
constexpr int kPer = 16 / (int)sizeof(E);
template <typename E>
__device__ __forceinline__ void unit_to_f(const uint4& u, float (&f)[kPer<E>]) {
  if constexpr (sizeof(E) == 2) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its float
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
}
template <typename E>
__device__ __forceinline__ uint4 f_to_unit(const float (&f)[kPer<E>]) {
  if constexpr (sizeof(E) == 2)
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  else
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// Elements of a row before its first 16-byte boundary (at most V).
template <typename E>
__device__ __forceinline__ int row_head(const E* row, int V) {
  return min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(E)));
}

struct RunningSum {
  float m = -INFINITY, s = 0.f;
  template <int N>
  __device__ __forceinline__ void add(const float (&z)[N], float c) {
    float mx = m;
#pragma unroll
    for (int i = 0; i < N; ++i) mx = fmaxf(mx, z[i]);
    const float a = anchor(mx);
    if (mx > m) {
      s *= ex2_approx((m - a) * c);
      m = mx;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s += ex2_approx((z[i] - a) * c);
  }
  __device__ __forceinline__ void merge(float m2, float s2, float c) {
    const float mx = fmaxf(m, m2), a = anchor(mx);
    s = s * ex2_approx((m - a) * c) + s2 * ex2_approx((m2 - a) * c);
    m = mx;
  }
};

template <typename E>
__global__ void __launch_bounds__(kRowThreads)
    distill_row_kernel(const E* __restrict__ logits, long long stride, const int32_t* __restrict__ ids,
                       const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                       float* __restrict__ token_loss, float* __restrict__ lse_out, float* __restrict__ part_loss,
                       int* __restrict__ part_count, unsigned* err) {
  __shared__ float s_m[kRowThreads / 32], s_s[kRowThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float c = kLog2e * inv_t;
  constexpr int P = kPer<E>, U = 4;
  float loss_acc = 0.f;
  int count = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const E* row = logits + (size_t)t * stride;
    const int32_t* id = ids + (size_t)t * K;
    const float* l = tl + (size_t)t * K;
    const bool mine = tid < K && usable_id(id[tid], l[tid], V, nullptr) >= 0;
    if (__syncthreads_or(mine)) {
      RunningSum r;
      const int head = row_head(row, V), units = (V - head) / P, tail = head + units * P;
      if (tid < head) r.add<1>({to_f(row[tid])}, c);
      const uint4* u4 = reinterpret_cast<const uint4*>(row + head);
      int u = tid;
      for (; u + (U - 1) * kRowThreads < units; u += U * kRowThreads) {
        uint4 w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) w[i] = __ldg(u4 + u + i * kRowThreads);
        float z[U * P];
#pragma unroll
        for (int i = 0; i < U; ++i) unit_to_f<E>(w[i], reinterpret_cast<float(&)[P]>(z[i * P]));
        r.add<U * P>(z, c);
      }
      for (; u < units; u += kRowThreads) {
        float z[P];
        unit_to_f<E>(__ldg(u4 + u), z);
        r.add<P>(z, c);
      }
      if (tail + tid < V) r.add<1>({to_f(row[tail + tid])}, c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, r.m, o), s2 = __shfl_xor_sync(0xffffffffu, r.s, o);
        r.merge(m2, s2, c);
      }
      if (lane == 0) {
        s_m[warp] = r.m;
        s_s[warp] = r.s;
      }
      __syncthreads();
      if (warp == 0) {
        RunningSum a;
        for (int w = 0; w < kRowThreads / 32; ++w) a.merge(s_m[w], s_s[w], c);
        const float lse = fmaf(anchor(a.m), inv_t, logf(a.s));
        const Teacher s = teacher_stats(id, l, K, V, inv_t, err);
        const float loss = row_loss(row, id, l, K, V, inv_t, temperature, s, lse);
        if (lane == 0) {
          token_loss[t] = loss;
          if (lse_out) lse_out[t] = lse;
        }
        loss_acc += loss;
        ++count;
      }
    } else if (warp == 0) {
      teacher_stats(id, l, K, V, inv_t, err);  // reports ids out of range
      if (lane == 0) {
        token_loss[t] = 0.f;
        if (lse_out) lse_out[t] = 0.f;
      }
    }
  }
  if (part_loss != nullptr && tid == 0) {
    part_loss[blockIdx.x] = loss_acc;
    part_count[blockIdx.x] = count;
  }
}

template <typename E>
__global__ void __launch_bounds__(kRowThreads)
    distill_bwd_row_kernel(const E* logits, long long stride, const int32_t* __restrict__ ids,
                           const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                           const float* __restrict__ lse_in, const int* __restrict__ loss_count, E* d_logits,
                           long long d_stride, unsigned* err) {
  __shared__ int s_id[kDistillMaxK];
  __shared__ float s_p[kDistillMaxK];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = loss_count ? *loss_count : 1;
  const float amp = n > 0 ? temperature / (float)n : 0.f;
  constexpr int P = kPer<E>, U = 4;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const E* row = logits + (size_t)t * stride;
    E* out = d_logits + (size_t)t * d_stride;
    const int32_t* id = ids + (size_t)t * K;
    const float* l = tl + (size_t)t * K;
    const int v = tid < K ? usable_id(id[tid], l[tid], V, err) : -1;
    const float zv = v >= 0 ? to_f(row[v]) : 0.f;  // before the row may be overwritten
    if (tid < K) s_id[tid] = v;
    const bool scored = __syncthreads_or(v >= 0) && amp != 0.f;
    const float lse = lse_in[t];
    // q of one value, times the amplitude
    auto grad = [&](float z) { return scored ? amp * ex2_approx(fmaf(z, inv_t, -lse) * kLog2e) : 0.f; };
    if (scored && warp == 0) {
      const Teacher s = teacher_stats(id, l, K, V, inv_t, nullptr);
      for (int k = lane; k < K; k += 32) s_p[k] = s_id[k] >= 0 ? expf(l[k] * inv_t - s.m) / s.sum : 0.f;
    }
    const int head = row_head(out, V);
    const bool together = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    if (together) {
      const int units = (V - head) / P, tail = head + units * P;
      if (tid < head) out[tid] = from_f<E>(grad(to_f(row[tid])));
      const uint4* src = reinterpret_cast<const uint4*>(row + head);
      uint4* dst = reinterpret_cast<uint4*>(out + head);
      int u = tid;
      for (; u + (U - 1) * kRowThreads < units; u += U * kRowThreads) {
        uint4 w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) w[i] = src[u + i * kRowThreads];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float z[P];
          unit_to_f<E>(w[i], z);
#pragma unroll
          for (int j = 0; j < P; ++j) z[j] = grad(z[j]);
          dst[u + i * kRowThreads] = f_to_unit<E>(z);
        }
      }
      for (; u < units; u += kRowThreads) {
        float z[P];
        unit_to_f<E>(src[u], z);
#pragma unroll
        for (int j = 0; j < P; ++j) z[j] = grad(z[j]);
        dst[u] = f_to_unit<E>(z);
      }
      if (tail + tid < V) out[tail + tid] = from_f<E>(grad(to_f(row[tail + tid])));
    } else {  // rows of the two buffers are aligned differently: value by value
      for (int i = tid; i < V; i += kRowThreads) out[i] = from_f<E>(grad(to_f(row[i])));
    }
    __syncthreads();
    if (scored && v >= 0) {
      // the first entry with this id takes the sum of all of them, in order
      float p = 0.f;
      bool first = true;
      for (int k = 0; k < K; ++k)
        if (s_id[k] == v) {
          if (k < tid) first = false;
          p += s_p[k];
        }
      if (first) out[v] = from_f<E>(amp * (ex2_approx(fmaf(zv, inv_t, -lse) * kLog2e) - p));
    }
    __syncthreads();  // s_id, s_p
  }
}

// Sum of the blocks' losses and scored rows, in block order per thread and a fixed tree.
__global__ void __launch_bounds__(256) distill_sum_kernel(const float* __restrict__ part_loss,
                                                          const int* __restrict__ part_count, int blocks,
                                                          float* loss_sum, int* count) {
  __shared__ double ss[256];
  __shared__ int sc[256];
  double s = 0.0;
  int n = 0;
  for (int i = threadIdx.x; i < blocks; i += 256) {
    s += (double)part_loss[i];
    n += part_count[i];
  }
  ss[threadIdx.x] = s;
  sc[threadIdx.x] = n;
  __syncthreads();
  for (int w = 128; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) {
      ss[threadIdx.x] += ss[threadIdx.x + w];
      sc[threadIdx.x] += sc[threadIdx.x + w];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    if (loss_sum) *loss_sum = (float)ss[0];
    if (count) *count = sc[0];
  }
}

// Blocks of a launch: resident blocks per SM of either form times the SMs, at most the rows.
int distill_blocks(int T, int V, int num_sms) {
  const int rows = V <= kWarpVocab ? (T + kWarpsPerBlock - 1) / kWarpsPerBlock : T;
  return std::max(1, std::min(rows, 8 * num_sms));
}

template <typename E>
void run_forward(const DistillArgs& a, int blocks, float* part_loss, int* part_count, cudaStream_t st) {
  const E* z = static_cast<const E*>(a.logits);
  const float inv_t = 1.f / a.temperature;
  auto warp_form = [&](auto kernel) {
    kernel<<<blocks, 32 * kWarpsPerBlock, 0, st>>>(z, a.stride, a.teacher_ids, a.teacher_logits, a.K, a.T, a.V,
                                                   a.temperature, inv_t, a.token_loss, a.lse, part_loss, part_count,
                                                   a.err);
  };
  if (a.V <= 32) warp_form(distill_warp_kernel<E, 1>);
  else if (a.V <= 64) warp_form(distill_warp_kernel<E, 2>);
  else if (a.V <= 128) warp_form(distill_warp_kernel<E, 4>);
  else if (a.V <= kWarpVocab) warp_form(distill_warp_kernel<E, 8>);
  else
    distill_row_kernel<E><<<blocks, kRowThreads, 0, st>>>(z, a.stride, a.teacher_ids, a.teacher_logits, a.K, a.T, a.V,
                                                          a.temperature, inv_t, a.token_loss, a.lse, part_loss,
                                                          part_count, a.err);
}

template <typename E>
void run_backward(const DistillArgs& a, int blocks, cudaStream_t st) {
  const E* z = static_cast<const E*>(a.logits);
  E* dz = static_cast<E*>(a.d_logits);
  const float inv_t = 1.f / a.temperature;
  auto launch = [&](auto kernel, int threads) {
    kernel<<<blocks, threads, 0, st>>>(z, a.stride, a.teacher_ids, a.teacher_logits, a.K, a.T, a.V, a.temperature,
                                       inv_t, a.lse, a.loss_count, dz, a.d_stride, a.err);
  };
  if (a.V <= 32) launch(distill_bwd_warp_kernel<E, 1>, 32 * kWarpsPerBlock);
  else if (a.V <= 64) launch(distill_bwd_warp_kernel<E, 2>, 32 * kWarpsPerBlock);
  else if (a.V <= 128) launch(distill_bwd_warp_kernel<E, 4>, 32 * kWarpsPerBlock);
  else if (a.V <= kWarpVocab) launch(distill_bwd_warp_kernel<E, 8>, 32 * kWarpsPerBlock);
  else launch(distill_bwd_row_kernel<E>, kRowThreads);
}

}  // namespace

size_t distill_workspace_bytes(int T, int V, int num_sms) { return 8 * (size_t)distill_blocks(T, V, num_sms); }

cudaError_t launch_distill_loss(const DistillArgs& a, float* loss_sum, int* count, void* workspace, int num_sms,
                                cudaStream_t st) {
  const bool want_sum = loss_sum != nullptr || count != nullptr;
  const int blocks = distill_blocks(a.T, a.V, num_sms);
  float* part_loss = want_sum ? static_cast<float*>(workspace) : nullptr;
  int* part_count = reinterpret_cast<int*>(part_loss + blocks);
  if (a.T > 0) {
    if (a.bf16) run_forward<__nv_bfloat16>(a, blocks, part_loss, part_count, st);
    else run_forward<float>(a, blocks, part_loss, part_count, st);
  }
  if (want_sum) distill_sum_kernel<<<1, 256, 0, st>>>(part_loss, part_count, a.T > 0 ? blocks : 0, loss_sum, count);
  return cudaGetLastError();
}

cudaError_t launch_distill_loss_backward(const DistillArgs& a, int num_sms, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  const int blocks = distill_blocks(a.T, a.V, num_sms);
  if (a.bf16) run_backward<__nv_bfloat16>(a, blocks, st);
  else run_backward<float>(a, blocks, st);
  return cudaGetLastError();
}

}  // namespace esm
