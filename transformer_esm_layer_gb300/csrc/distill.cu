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
// A row without a usable entry is not scored: loss, lse and gradient 0, whatever its logits (the loss
// leaves them unread in rows above 256 values).
// Logits are read once per call (forward: running maximum and sum per thread, merged in a
// fixed order; backward: q from the forward's lse, each value overwritten where it is read, so
// the gradient may take the logits' place).  Exponentials, sums and the loss are fp32 whatever
// the logits' type; the gradient is rounded once, to the logits' type.
//
// Both directions are bound by the logits' bytes; a row too short for that is bound by the
// latency of its chain of loads and shuffles.  Three forms (rows_form below chooses): G lanes per
// row with the row in registers, a warp per row, a block per row.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace esm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kGroupVocab = 256;   // up to here the row is held in registers
constexpr int kThreads = 256;      // of every block
constexpr int kWarps = kThreads / 32;
constexpr int kRowUnits = 4;       // 16-byte units of a row that a thread loads at once
constexpr int kFewEntries = 32;    // entries of a row up to which each is compared with all
constexpr int kRowBlocks = 4;      // resident blocks per SM of the streaming forms
static_assert(kDistillMaxK <= kThreads, "one teacher entry per thread in the block form");
static_assert(kDistillMaxK <= 32 * 8, "at most eight teacher entries per lane in the warp form");

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

// Sum and maximum over the G lanes of a group (G consecutive lanes, a power of two).
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
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

// Block partial sums of the losses and scored rows: the warps' in order.
__device__ __forceinline__ void write_partials(float loss, int count, float* part_loss, int* part_count) {
  __shared__ float s_loss[kWarps];
  __shared__ int s_count[kWarps];
  if (part_loss == nullptr) return;
  loss = group_sum<32>(loss);
  count = __reduce_add_sync(0xffffffffu, count);
  if ((threadIdx.x & 31) == 0) {
    s_loss[threadIdx.x >> 5] = loss;
    s_count[threadIdx.x >> 5] = count;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float a = 0.f;
    int n = 0;
    for (int w = 0; w < kWarps; ++w) {
      a += s_loss[w];
      n += s_count[w];
    }
    part_loss[blockIdx.x] = a;
    part_count[blockIdx.x] = n;
  }
}

// ---------------------------------------------------------------- group form
// G lanes per row, N values of it per lane.  All loads of a row but the student's logits at the
// teacher's ids are issued together; with 8 lanes per row the reductions are three shuffles
// deep, and a warp has four rows' chains in flight (16384 x 33 fp32, 8 entries: loss 8.9 us and
// gradient 8.9 us a call against 15.0 and 17.0 with a warp per row, measured as at rows_form).
//
// Teacher softmax of the group's row, entries k = lane of the group, + G, ...: the maximum m of l (0 if
// there is no finite one), the sum of exp((l - m) / t), whether any entry is usable.  The
// difference is taken before the division: a lowest float divided by t < 1 would be -inf.
struct Teacher {
  float m, sum;
  bool any;
};
template <int G>
__device__ __forceinline__ Teacher teacher_stats(const int32_t* ids, const float* tl, int K, int V, float inv_t,
                                                 unsigned* err) {
  const int lane = threadIdx.x & 31, gl = lane & (G - 1);
  Teacher s{-INFINITY, 0.f, false};
  for (int k = gl; k < K; k += G) {
    if (usable_id(ids[k], tl[k], V, err) < 0) continue;
    s.m = fmaxf(s.m, tl[k]);
    s.any = true;
  }
  s.m = anchor(group_max<G>(s.m));
  constexpr unsigned kGroup = G == 32 ? 0xffffffffu : (1u << G) - 1u;
  s.any = (__ballot_sync(0xffffffffu, s.any) >> (lane - gl) & kGroup) != 0u;
  for (int k = gl; k < K; k += G)
    if (usable_id(ids[k], tl[k], V, nullptr) >= 0) s.sum += expf((tl[k] - s.m) * inv_t);
  s.sum = group_sum<G>(s.sum);
  return s;
}

template <typename E, int G, int N>
__global__ void __launch_bounds__(kThreads)
    distill_group_kernel(const E* __restrict__ logits, long long stride, const int32_t* __restrict__ ids,
                         const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                         float* __restrict__ token_loss, float* __restrict__ lse_out, float* __restrict__ part_loss,
                         int* __restrict__ part_count, unsigned* err) {
  constexpr int R = kThreads / G;  // rows of a block
  const int lane = threadIdx.x & 31, gl = lane & (G - 1);
  const float c = kLog2e * inv_t;
  float loss_acc = 0.f;
  int count = 0;
  // (a group past the last row follows its warp with that row and writes nothing)
  for (int t0 = blockIdx.x * R + (threadIdx.x >> 5) * (32 / G); t0 < T; t0 += gridDim.x * R) {
    const bool live = t0 + lane / G < T;
    const int t = min(t0 + lane / G, T - 1);
    const E* row = logits + (size_t)t * stride;
    const int32_t* id = ids + (size_t)t * K;
    const float* l = tl + (size_t)t * K;
    float z[N];
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = gl + G * i < V ? to_f(row[gl + G * i]) : -INFINITY;
    const Teacher s = teacher_stats<G>(id, l, K, V, inv_t, err);
    float m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, z[i]);
    m = anchor(group_max<G>(m));
#pragma unroll
    for (int i = 0; i < N; ++i) sum += ex2_approx((z[i] - m) * c);
    const float lse = fmaf(m, inv_t, logf(group_sum<G>(sum)));
    const float log_sum = logf(s.sum), inv_sum = 1.f / s.sum;
    float loss = 0.f;
    for (int k = gl; k < K; k += G) {
      const int v = usable_id(id[k], l[k], V, nullptr);
      if (v < 0) continue;
      const float a = (l[k] - s.m) * inv_t, p = expf(a) * inv_sum;
      // an entry whose probability underflows adds nothing, whatever the student makes of it
      if (p != 0.f) loss = fmaf(p, (a - log_sum) - (to_f(row[v]) * inv_t - lse), loss);
    }
    loss = temperature * temperature * group_sum<G>(loss);
    if (live && gl == 0) {
      token_loss[t] = s.any ? loss : 0.f;
      if (lse_out) lse_out[t] = s.any ? lse : 0.f;
      if (s.any) {
        loss_acc += loss;
        ++count;
      }
    }
  }
  write_partials(loss_acc, count, part_loss, part_count);
}

template <typename E, int G, int N>
__global__ void __launch_bounds__(kThreads)
    distill_bwd_group_kernel(const E* logits, long long stride, const int32_t* __restrict__ ids,
                             const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                             const float* __restrict__ lse_in, const int* __restrict__ loss_count, E* d_logits,
                             long long d_stride, unsigned* err) {
  constexpr int R = kThreads / G;
  __shared__ float s_p[R][G * N];
  const int lane = threadIdx.x & 31, gl = lane & (G - 1);
  float* p_row = s_p[threadIdx.x / G];
  for (int t0 = blockIdx.x * R + (threadIdx.x >> 5) * (32 / G); t0 < T; t0 += gridDim.x * R) {
    const bool live = t0 + lane / G < T;
    const int t = min(t0 + lane / G, T - 1);
    const E* row = logits + (size_t)t * stride;
    E* out = d_logits + (size_t)t * d_stride;
    const int32_t* id = ids + (size_t)t * K;
    const float* l = tl + (size_t)t * K;
    float z[N];
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = live && gl + G * i < V ? to_f(row[gl + G * i]) : 0.f;
    const float lse = lse_in[t];
    const int n = loss_count ? *loss_count : 1;
    const Teacher s = teacher_stats<G>(id, l, K, V, inv_t, err);
    const float amp = s.any && n > 0 ? temperature / (float)n : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) p_row[gl + G * i] = 0.f;
    __syncwarp();
    const float inv_sum = 1.f / s.sum;
    for (int k0 = 0; k0 < K; k0 += G) {
      const int k = k0 + gl;
      const int v = k < K ? usable_id(id[k], l[k], V, nullptr) : -1;
      const float p = v >= 0 ? expf((l[k] - s.m) * inv_t) * inv_sum : 0.f;
      // (the key tells the rows of a warp apart, and unused entries)
      const unsigned same = __match_any_sync(0xffffffffu, v >= 0 ? (lane - gl) * kGroupVocab + v : -1 - lane);
      if (__any_sync(0xffffffffu, (same & (same - 1)) != 0u)) {
        // an id stands in a row twice: one entry after the other
        for (int j = 0; j < G; ++j) {
          if (gl == j && v >= 0) p_row[v] += p;
          __syncwarp();
        }
      } else if (v >= 0) {
        p_row[v] += p;
      }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = gl + G * i;
      if (live && v < V) {
        const float q = ex2_approx(fmaf(z[i], inv_t, -lse) * kLog2e);
        out[v] = from_f<E>(amp == 0.f ? 0.f : amp * (q - p_row[v]));
      }
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- warp and block forms
// W warps per row (1 or kWarps), EN teacher entries per thread.  The forward loads the next
// kRowUnits units of each thread before it works on the present ones, which keeps 64 bytes per
// thread in flight through the exponentials (8192 x 32000 bf16: 5.7 TB/s; loads and work in
// turn 4.7).
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

// Running maximum and sum of exponentials of z / t: the sum is relative to the maximum.
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
    if constexpr (N % 2 == 0) {  // two values per f32x2 instruction
      const uint64_t a2 = f2_pack(-a, -a), c2 = f2_pack(c, c);
      uint64_t sum = f2_pack(s, 0.f);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float x, y;
        f2_unpack(f2_mul(f2_add(f2_pack(z[i], z[i + 1]), a2), c2), x, y);
        sum = f2_add(sum, f2_pack(ex2_approx(x), ex2_approx(y)));
      }
      float x, y;
      f2_unpack(sum, x, y);
      s = x + y;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) s += ex2_approx((z[i] - a) * c);
    }
  }
  __device__ __forceinline__ void merge(float m2, float s2, float c) {
    const float mx = fmaxf(m, m2), a = anchor(mx);
    s = s * ex2_approx((m - a) * c) + s2 * ex2_approx((m2 - a) * c);
    m = mx;
  }
};

// The teacher's side of a row's loss over some of its entries, relative to their maximum m: with
// a = (l - m) / t, s = sum exp(a), x = sum exp(a) (a - z / t).  Then loss / t^2 = x / s - log s + lse.
struct TeacherSum {
  float m = -INFINITY, s = 0.f, x = 0.f;
  __device__ __forceinline__ void merge(float m2, float s2, float x2, float inv_t) {
    const float mx = anchor(fmaxf(m, m2)), a = (m - mx) * inv_t, b = (m2 - mx) * inv_t;
    const float f = m == -INFINITY ? 0.f : expf(a), g = m2 == -INFINITY ? 0.f : expf(b);
    // a part whose weight underflows adds nothing, whatever the student makes of its entries
    x = (f != 0.f ? f * fmaf(s, a, x) : 0.f) + (g != 0.f ? g * fmaf(s2, b, x2) : 0.f);
    s = f * s + g * s2;
    m = fmaxf(m, m2);
  }
};

// Any of the row's threads, and a barrier: what they read or wrote before is ordered with what they
// write or read after it (a vote alone does not order memory).
template <int W>
__device__ __forceinline__ bool row_any(bool v) {
  if constexpr (W == 1) {
    const bool any = __any_sync(0xffffffffu, v);
    __syncwarp();
    return any;
  } else {
    return __syncthreads_or(v);
  }
}
template <int W>
__device__ __forceinline__ void row_sync() {
  if constexpr (W == 1) __syncwarp();
  else __syncthreads();
}

// The ids and logits of the entries are fetched a row ahead, and the student's logits at the
// ids before the row is streamed, so that nothing waits for a load once the row has been read.
template <typename E, int W, int EN>
__global__ void __launch_bounds__(kThreads, EN > 2 ? 2 : kRowBlocks)
    distill_row_kernel(const E* __restrict__ logits, long long stride, const int32_t* __restrict__ ids,
                       const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                       float* __restrict__ token_loss, float* __restrict__ lse_out, float* __restrict__ part_loss,
                       int* __restrict__ part_count, unsigned* err) {
  constexpr int P = kPer<E>, U = kRowUnits, RT = 32 * W, R = kThreads / RT;
  __shared__ float s_part[5][kWarps];
  const int tid = threadIdx.x % RT, warp = tid >> 5, lane = tid & 31;
  const float c = kLog2e * inv_t;
  const uint32_t kNone = sizeof(E) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
  float loss_acc = 0.f;
  int count = 0, id_next[EN];
  float l_next[EN];
  auto fetch = [&](int t) {
#pragma unroll
    for (int e = 0; e < EN; ++e) {
      const int k = tid + RT * e;
      id_next[e] = -1;
      l_next[e] = 0.f;
      if (t < T && k < K) {
        id_next[e] = __ldg(ids + (size_t)t * K + k);
        l_next[e] = __ldg(tl + (size_t)t * K + k);
      }
    }
  };
  const int first = blockIdx.x * R + threadIdx.x / RT, step = gridDim.x * R;
  fetch(first);
  for (int t = first; t < T; t += step) {
    const E* row = logits + (size_t)t * stride;
    int id[EN];
    float l[EN];
    bool mine = false;
#pragma unroll
    for (int e = 0; e < EN; ++e) {
      l[e] = l_next[e];
      id[e] = usable_id(id_next[e], l[e], V, err);
      mine |= id[e] >= 0;
    }
    fetch(t + step);
    if (!row_any<W>(mine)) {
      if (tid == 0) {
        token_loss[t] = 0.f;
        if (lse_out) lse_out[t] = 0.f;
      }
      continue;
    }
    float zk[EN];
#pragma unroll
    for (int e = 0; e < EN; ++e) zk[e] = id[e] >= 0 ? to_f(row[id[e]]) : 0.f;
    RunningSum r;
    const int head = row_head(row, V), units = (V - head) / P, tail = head + units * P;
    if (tid < head) r.add<1>({to_f(row[tid])}, c);
    const uint4* u4 = reinterpret_cast<const uint4*>(row + head);
    uint4 w[U];
    auto load = [&](int u) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        w[i] = u + i * RT < units ? __ldg(u4 + u + i * RT) : make_uint4(kNone, kNone, kNone, kNone);
    };
    load(tid);
    for (int u = tid; u < units; u += U * RT) {
      float z[U * P];
      uint4 x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) x[i] = w[i];
      load(u + U * RT);
#pragma unroll
      for (int i = 0; i < U; ++i) unit_to_f<E>(x[i], reinterpret_cast<float(&)[P]>(z[i * P]));
      r.add<U * P>(z, c);
    }
    if (tail + tid < V) r.add<1>({to_f(row[tail + tid])}, c);
    // this warp's entries
    TeacherSum s;
    bool here = false;
#pragma unroll
    for (int e = 0; e < EN; ++e)
      if (id[e] >= 0) {
        s.m = fmaxf(s.m, l[e]);
        here = true;
      }
    if (__any_sync(0xffffffffu, here)) {
      s.m = group_max<32>(s.m);
#pragma unroll
      for (int e = 0; e < EN; ++e) {
        const float a = (l[e] - anchor(s.m)) * inv_t, w = id[e] >= 0 ? expf(a) : 0.f;
        s.s += w;
        if (w != 0.f) s.x = fmaf(w, a - zk[e] * inv_t, s.x);
      }
      s.s = group_sum<32>(s.s);
      s.x = group_sum<32>(s.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, r.m, o), s2 = __shfl_xor_sync(0xffffffffu, r.s, o);
      r.merge(m2, s2, c);
    }
    if constexpr (W > 1) {
      if (lane == 0) {
        s_part[0][warp] = r.m;
        s_part[1][warp] = r.s;
        s_part[2][warp] = s.m;
        s_part[3][warp] = s.s;
        s_part[4][warp] = s.x;
      }
      __syncthreads();
      if (warp > 0) continue;  // (the next row's barrier keeps s_part until warp 0 has read it)
      const int w = lane & (W - 1);
      r.m = s_part[0][w];
      r.s = s_part[1][w];
      s.m = s_part[2][w];
      s.s = s_part[3][w];
      s.x = s_part[4][w];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, r.m, o), s2 = __shfl_xor_sync(0xffffffffu, r.s, o);
        r.merge(m2, s2, c);
        const float tm = __shfl_xor_sync(0xffffffffu, s.m, o), ts = __shfl_xor_sync(0xffffffffu, s.s, o);
        const float tx = __shfl_xor_sync(0xffffffffu, s.x, o);
        s.merge(tm, ts, tx, inv_t);
      }
    }
    if (lane == 0) {
      const float lse = fmaf(anchor(r.m), inv_t, logf(r.s));
      const float loss = temperature * temperature * ((s.x / s.s - logf(s.s)) + lse);
      token_loss[t] = loss;
      if (lse_out) lse_out[t] = lse;
      loss_acc += loss;
      ++count;
    }
  }
  if constexpr (W > 1) __syncthreads();
  write_partials(loss_acc, count, part_loss, part_count);
}

// A small number in a value's place, among threads that synchronise in between.
template <typename E>
__device__ __forceinline__ void put_bits(E* p, int n) {
  if constexpr (sizeof(E) == 2) *reinterpret_cast<volatile unsigned short*>(p) = (unsigned short)n;
  else *reinterpret_cast<volatile int*>(p) = n;
}
template <typename E>
__device__ __forceinline__ int get_bits(const E* p) {
  if constexpr (sizeof(E) == 2) return *reinterpret_cast<const volatile unsigned short*>(p);
  else return *reinterpret_cast<const volatile int*>(p);
}

template <typename E, int W, int EN>
__global__ void __launch_bounds__(kThreads)
    distill_bwd_row_kernel(const E* logits, long long stride, const int32_t* __restrict__ ids,
                           const float* __restrict__ tl, int K, int T, int V, float temperature, float inv_t,
                           const float* __restrict__ lse_in, const int* __restrict__ loss_count, E* d_logits,
                           long long d_stride, unsigned* err) {
  constexpr int P = kPer<E>, U = kRowUnits, RT = 32 * W, R = kThreads / RT;
  __shared__ int s_id_all[R][RT * EN];
  __shared__ float s_p_all[R][RT * EN];
  const int tid = threadIdx.x % RT, warp = tid >> 5, lane = tid & 31;
  int* s_id = s_id_all[threadIdx.x / RT];
  float* s_p = s_p_all[threadIdx.x / RT];
  const int n = loss_count ? *loss_count : 1;
  const float amp = n > 0 ? temperature / (float)n : 0.f;
  for (int t = blockIdx.x * R + threadIdx.x / RT; t < T; t += gridDim.x * R) {
    const E* row = logits + (size_t)t * stride;
    E* out = d_logits + (size_t)t * d_stride;
    const int32_t* id = ids + (size_t)t * K;
    const float* l = tl + (size_t)t * K;
    int v[EN];
    float zv[EN];
    bool mine = false;
#pragma unroll
    for (int e = 0; e < EN; ++e) {
      const int k = tid + RT * e;
      v[e] = k < K ? usable_id(id[k], l[k], V, err) : -1;
      zv[e] = v[e] >= 0 ? to_f(row[v[e]]) : 0.f;  // before the row may be overwritten
      mine |= v[e] >= 0;
      if (k < K) s_id[k] = v[e];
    }
    const bool scored = row_any<W>(mine) && amp != 0.f;
    const float lse = lse_in[t];
    // q of one value, times the amplitude
    auto grad = [&](float z) { return scored ? amp * ex2_approx(fmaf(z, inv_t, -lse) * kLog2e) : 0.f; };
    if (scored && warp == 0) {
      const Teacher s = teacher_stats<32>(id, l, K, V, inv_t, nullptr);
      for (int k = lane; k < K; k += 32) s_p[k] = s_id[k] >= 0 ? expf((l[k] - s.m) * inv_t) / s.sum : 0.f;
    }
    const int head = row_head(out, V);
    const bool together = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    if (together) {
      const int units = (V - head) / P, tail = head + units * P;
      if (tid < head) out[tid] = from_f<E>(grad(to_f(row[tid])));
      const uint4* src = reinterpret_cast<const uint4*>(row + head);
      uint4* dst = reinterpret_cast<uint4*>(out + head);
      for (int u = tid; u < units; u += U * RT) {
        uint4 w[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (u + i * RT < units) w[i] = src[u + i * RT];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (u + i * RT >= units) break;
          float z[P];
          unit_to_f<E>(w[i], z);
#pragma unroll
          for (int j = 0; j < P; ++j) z[j] = grad(z[j]);
          dst[u + i * RT] = f_to_unit<E>(z);
        }
      }
      if (tail + tid < V) out[tail + tid] = from_f<E>(grad(to_f(row[tail + tid])));
    } else {  // rows of the two buffers are aligned differently: value by value
      for (int i = tid; i < V; i += RT) out[i] = from_f<E>(grad(to_f(row[i])));
    }
    row_sync<W>();
    if (scored) {
      // Many entries: each leaves its number where its value goes, and one that finds another's
      // shares its id.  Ids of a row are nearly always distinct, and then this replaces comparing
      // each with all (65536 x 1000 bf16, 100 entries: 222 us against 388; with 16 entries the
      // comparisons are faster, 71 us against 78; measured as at rows_form).
      bool shared = K <= kFewEntries;
      if (!shared) {
#pragma unroll
        for (int e = 0; e < EN; ++e)
          if (v[e] >= 0) put_bits(out + v[e], tid + RT * e);
        row_sync<W>();
#pragma unroll
        for (int e = 0; e < EN; ++e)
          if (v[e] >= 0) shared |= get_bits(out + v[e]) != tid + RT * e;
      }
      float p[EN];
      bool is_first[EN];
#pragma unroll
      for (int e = 0; e < EN; ++e) {
        is_first[e] = v[e] >= 0;
        p[e] = is_first[e] ? s_p[tid + RT * e] : 0.f;
      }
      if (row_any<W>(shared)) {
        // the first entry with an id takes the sum of all of them, in order
#pragma unroll
        for (int e = 0; e < EN; ++e) p[e] = 0.f;
        for (int k = 0; k < K; ++k) {
          const int other = s_id[k];
          const float pk = s_p[k];
#pragma unroll
          for (int e = 0; e < EN; ++e)
            if (other == v[e]) {
              if (k < tid + RT * e) is_first[e] = false;
              p[e] += pk;
            }
        }
      }
#pragma unroll
      for (int e = 0; e < EN; ++e)
        if (is_first[e]) out[v[e]] = from_f<E>(amp * (ex2_approx(fmaf(zv[e], inv_t, -lse) * kLog2e) - p[e]));
    }
    row_sync<W>();  // s_id, s_p
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

// The form of a call, as the threads of a row: 8, 16 or 32 lanes with the row in registers; a warp
// (with 2 or 8 teacher entries per lane) or a block that streams it.  A warp per row keeps eight
// times the rows in flight: it is taken when there are more rows than resident blocks, unless
// they are long.  Warp and block per row, loss (without its sums) and gradient in us, each call by
// events after an L2 flush, with 16 to 32 entries: 2000 rows of 8 KB 13.0 / 15.0 and 17.1 / 19.1;
// 65536 x 1000 bf16 56 / 70 and 257 / 322; 2000 rows of 32 KB 25.2 / 33.4 and 23.2 / 31.5, of 64 KB
// 41.6 / 55.9 and 35.5 / 51.9; 300 rows of 16 KB 12.9 / 15.0 and 8.9 / 10.9.
enum class Form { kGroup8x4, kGroup8x8, kGroup16x8, kGroup32x8, kWarpRow2, kWarpRow8, kBlockRow };
constexpr int kWarpRowBytes = 32768;
Form rows_form(int T, int V, int K, int elem, int num_sms) {
  if (V <= 32) return Form::kGroup8x4;
  if (V <= 64) return Form::kGroup8x8;
  if (V <= 128) return Form::kGroup16x8;
  if (V <= kGroupVocab) return Form::kGroup32x8;
  if (T <= kRowBlocks * num_sms || (long long)V * elem > kWarpRowBytes) return Form::kBlockRow;
  return K <= 64 ? Form::kWarpRow2 : Form::kWarpRow8;
}
int form_rows(Form f) {  // rows of a block
  switch (f) {
    case Form::kGroup8x4:
    case Form::kGroup8x8: return kThreads / 8;
    case Form::kGroup16x8: return kThreads / 16;
    case Form::kBlockRow: return 1;
    default: return kWarps;
  }
}

// Blocks of a launch: those resident at once (the group forms' registers let more in), at most
// the rows'.
int distill_blocks(int T, Form f, int num_sms) {
  const int r = form_rows(f), per_sm = f < Form::kWarpRow2 ? 2 * kRowBlocks : kRowBlocks;
  return std::max(1, std::min((T + r - 1) / r, per_sm * num_sms));
}

template <typename E>
void run_forward(const DistillArgs& a, Form f, int blocks, float* part_loss, int* part_count, cudaStream_t st) {
  const E* z = static_cast<const E*>(a.logits);
  const float inv_t = 1.f / a.temperature;
  auto launch = [&](auto kernel) {
    kernel<<<blocks, kThreads, 0, st>>>(z, a.stride, a.teacher_ids, a.teacher_logits, a.K, a.T, a.V, a.temperature,
                                        inv_t, a.token_loss, a.lse, part_loss, part_count, a.err);
  };
  switch (f) {
    case Form::kGroup8x4: return launch(distill_group_kernel<E, 8, 4>);
    case Form::kGroup8x8: return launch(distill_group_kernel<E, 8, 8>);
    case Form::kGroup16x8: return launch(distill_group_kernel<E, 16, 8>);
    case Form::kGroup32x8: return launch(distill_group_kernel<E, 32, 8>);
    case Form::kWarpRow2: return launch(distill_row_kernel<E, 1, 2>);
    case Form::kWarpRow8: return launch(distill_row_kernel<E, 1, 8>);
    case Form::kBlockRow: return launch(distill_row_kernel<E, kWarps, 1>);
  }
}

template <typename E>
void run_backward(const DistillArgs& a, Form f, int blocks, cudaStream_t st) {
  const E* z = static_cast<const E*>(a.logits);
  const float inv_t = 1.f / a.temperature;
  auto launch = [&](auto kernel) {
    kernel<<<blocks, kThreads, 0, st>>>(z, a.stride, a.teacher_ids, a.teacher_logits, a.K, a.T, a.V, a.temperature,
                                        inv_t, a.lse, a.loss_count, static_cast<E*>(a.d_logits), a.d_stride, a.err);
  };
  switch (f) {
    case Form::kGroup8x4: return launch(distill_bwd_group_kernel<E, 8, 4>);
    case Form::kGroup8x8: return launch(distill_bwd_group_kernel<E, 8, 8>);
    case Form::kGroup16x8: return launch(distill_bwd_group_kernel<E, 16, 8>);
    case Form::kGroup32x8: return launch(distill_bwd_group_kernel<E, 32, 8>);
    case Form::kWarpRow2: return launch(distill_bwd_row_kernel<E, 1, 2>);
    case Form::kWarpRow8: return launch(distill_bwd_row_kernel<E, 1, 8>);
    case Form::kBlockRow: return launch(distill_bwd_row_kernel<E, kWarps, 1>);
  }
}

}  // namespace

// (for any number of entries and either type: the block form's count is the largest)
size_t distill_workspace_bytes(int T, int V, int num_sms) {
  const int most = V <= kGroupVocab ? distill_blocks(T, rows_form(T, V, 1, 4, num_sms), num_sms)
                                    : distill_blocks(T, Form::kBlockRow, num_sms);
  return 8 * (size_t)most;
}

cudaError_t launch_distill_loss(const DistillArgs& a, float* loss_sum, int* count, void* workspace, int num_sms,
                                cudaStream_t st) {
  const bool want_sum = loss_sum != nullptr || count != nullptr;
  const Form f = rows_form(a.T, a.V, a.K, a.bf16 ? 2 : 4, num_sms);
  const int blocks = distill_blocks(a.T, f, num_sms);
  float* part_loss = want_sum ? static_cast<float*>(workspace) : nullptr;
  int* part_count = want_sum ? reinterpret_cast<int*>(part_loss + blocks) : nullptr;
  if (a.T > 0) {
    if (a.bf16) run_forward<__nv_bfloat16>(a, f, blocks, part_loss, part_count, st);
    else run_forward<float>(a, f, blocks, part_loss, part_count, st);
  }
  if (want_sum) distill_sum_kernel<<<1, 256, 0, st>>>(part_loss, part_count, a.T > 0 ? blocks : 0, loss_sum, count);
  return cudaGetLastError();
}

cudaError_t launch_distill_loss_backward(const DistillArgs& a, int num_sms, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  const Form f = rows_form(a.T, a.V, a.K, a.bf16 ? 2 : 4, num_sms);
  const int blocks = distill_blocks(a.T, f, num_sms);
  if (a.bf16) run_backward<__nv_bfloat16>(a, f, blocks, st);
  else run_backward<float>(a, f, blocks, st);
  return cudaGetLastError();
}

}  // namespace esm
