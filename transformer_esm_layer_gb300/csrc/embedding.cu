// Embedding lookup with scaling and dropout, and its gradient:
//   out[t] = keep(t, c) * drop_scale * scale * row_scale[t] * table[id_t]     (id -1: zeros)
//   d_table[v] (+)= scale * sum over t with id_t = v of row_scale[t] * keep(t, c) * drop_scale * d_out[t]
// The sums run in a fixed order, so results do not depend on scheduling.
//
// Bound by memory: the rows met and the output; for the gradient d_out and the table's rows.
#include <algorithm>

#include "dropout.cuh"
#include "internal.h"

namespace esm {
namespace {

// An id that has a row, or -1; other ids latch ERRBIT_TOKEN.
__device__ __forceinline__ int checked_id(const EmbedArgs& a, int t, bool report) {
  const int id = __ldg(a.ids + t);
  if (id >= 0 && id < a.vocab) return id;
  if (id != -1 && report) latch_error(a.err, ERRBIT_TOKEN);
  return -1;
}

__device__ __forceinline__ float token_scale(const EmbedArgs& a, int t) {
  return a.row_scale ? a.scale * __ldg(a.row_scale + t) : a.scale;
}

// One warp per 256 columns of a token.
template <typename TE, typename TO, bool VEC>
__global__ void __launch_bounds__(256) embed_scaled_kernel(const EmbedArgs a) {
  const PhiloxState ps = philox_state(a.mask);
  const int lane = threadIdx.x & 31;
  const long long spans = (a.cols + 255) / 256, per_row = (a.cols + 7) / 8, total = spans * a.tokens;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
    const int t = (int)(i / spans);
    const long long c0 = (i - t * spans) * 256;
    const int left = (int)min((long long)256, a.cols - c0);
    const int id = checked_id(a, t, lane == 0 && c0 == 0);
    float v[8];
    if (id >= 0) {
      span_load<VEC>(static_cast<const TE*>(a.table) + (long long)id * a.cols + c0, left, lane, v);
      const float f = token_scale(a, t);
      const uint32_t keep = span_keep<VEC>(a.mask, ps, (unsigned long long)(t * per_row + c0 / 8), lane);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = keep >> k & 1u ? v[k] * f * a.mask.scale : 0.f;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.f;
    }
    span_store<VEC>(static_cast<TO*>(a.out) + t * a.out_stride + c0, left, lane, v);
  }
}

// One warp per id and 256 columns: it looks through all tokens, 32 at a time.
template <typename TO, bool VEC>
__global__ void __launch_bounds__(256) embed_grad_kernel(const EmbedArgs a) {
  const PhiloxState ps = philox_state(a.mask);
  const int lane = threadIdx.x & 31;
  const long long spans = (a.cols + 255) / 256, per_row = (a.cols + 7) / 8, total = spans * a.vocab;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
    const int v = (int)(i / spans);
    const long long c0 = (i - v * spans) * 256;
    const int left = (int)min((long long)256, a.cols - c0);
    float* dst = a.d_table + (long long)v * a.cols + c0;
    float acc[8] = {};
    if (a.accumulate) span_load<VEC>(dst, left, lane, acc);
    for (int t0 = 0; t0 < a.tokens; t0 += 32) {
      const int t = t0 + lane;
      const int id = t < a.tokens ? checked_id(a, t, i == 0) : -1;
      for (uint32_t hit = __ballot_sync(0xffffffffu, id == v); hit; hit &= hit - 1) {
        const int m = t0 + __ffs(hit) - 1;
        float g[8];
        span_load<VEC>(static_cast<const TO*>(a.out) + m * a.out_stride + c0, left, lane, g);
        const float f = token_scale(a, m);
        const uint32_t keep = span_keep<VEC>(a.mask, ps, (unsigned long long)(m * per_row + c0 / 8), lane);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += keep >> k & 1u ? g[k] * f * a.mask.scale : 0.f;
      }
    }
    span_store<VEC>(dst, left, lane, acc);
  }
}

unsigned warps_grid(long long warps, int num_sms) {
  return (unsigned)std::min((warps + 7) / 8, (long long)num_sms * 64);
}

template <typename TE, typename TO>
void launch_lookup(const EmbedArgs& a, int num_sms, cudaStream_t st) {
  const unsigned grid = warps_grid((a.cols + 255) / 256 * (long long)a.tokens, num_sms);
  if (rows_on_16(a.table, a.cols, sizeof(TE)) && rows_on_16(a.out, a.out_stride, sizeof(TO)))
    embed_scaled_kernel<TE, TO, true><<<grid, 256, 0, st>>>(a);
  else
    embed_scaled_kernel<TE, TO, false><<<grid, 256, 0, st>>>(a);
}

template <typename TO>
void launch_grad(const EmbedArgs& a, int num_sms, cudaStream_t st) {
  const unsigned grid = warps_grid((a.cols + 255) / 256 * (long long)a.vocab, num_sms);
  if (rows_on_16(a.d_table, a.cols, 4) && rows_on_16(a.out, a.out_stride, sizeof(TO)))
    embed_grad_kernel<TO, true><<<grid, 256, 0, st>>>(a);
  else
    embed_grad_kernel<TO, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_embed_scaled(const EmbedArgs& a, int num_sms, cudaStream_t st) {
  if (a.tokens <= 0) return cudaSuccess;
  using bf16 = __nv_bfloat16;
  if (a.table_bf16) {
    if (a.out_bf16) launch_lookup<bf16, bf16>(a, num_sms, st);
    else launch_lookup<bf16, float>(a, num_sms, st);
  } else {
    if (a.out_bf16) launch_lookup<float, bf16>(a, num_sms, st);
    else launch_lookup<float, float>(a, num_sms, st);
  }
  return cudaGetLastError();
}

size_t embed_grad_workspace_bytes(int tokens, int vocab, int cols, int num_sms) { return 256; }

cudaError_t launch_embed_grad(const EmbedArgs& a, void* workspace, int num_sms, cudaStream_t st) {
  if (a.out_bf16) launch_grad<__nv_bfloat16>(a, num_sms, st);
  else launch_grad<float>(a, num_sms, st);
  return cudaGetLastError();
}

}  // namespace esm
