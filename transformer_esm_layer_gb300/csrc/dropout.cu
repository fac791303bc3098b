// Dropout whose mask is drawn again wherever it is needed and never stored (see dropout.cuh):
//   y = [residual +] keep(r, c) * scale * x
// The gradient is the same call on dy.
//
// Bound by memory: x (and the residual) read once, y written once.
#include <algorithm>

#include "dropout.cuh"
#include "internal.h"

namespace esm {
namespace {

// One warp per 256 columns of a row, in a grid-stride loop.
template <typename TX, typename TY, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutArgs a) {
  const PhiloxState ps = philox_state(a.mask);
  const int lane = threadIdx.x & 31;
  const long long spans = (a.cols + 255) / 256, per_row = (a.cols + 7) / 8, total = spans * a.rows;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
    const long long r = i / spans;
    const long long c0 = (i - r * spans) * 256;
    const int left = (int)min((long long)256, a.cols - c0);
    float x[8], res[8];
    span_load<VEC>(static_cast<const TX*>(a.x) + r * a.x_stride + c0, left, lane, x);
    if (a.residual) span_load<VEC>(static_cast<const TY*>(a.residual) + r * a.res_stride + c0, left, lane, res);
    const uint32_t keep = span_keep<VEC>(a.mask, ps, (unsigned long long)(r * per_row + c0 / 8), lane);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = keep >> k & 1u ? x[k] * a.mask.scale : 0.f;
      if (a.residual) x[k] += res[k];
    }
    span_store<VEC>(static_cast<TY*>(a.y) + r * a.y_stride + c0, left, lane, x);
  }
}

template <typename TX, typename TY>
void launch(const DropoutArgs& a, bool vec, int num_sms, cudaStream_t st) {
  const long long warps = (a.cols + 255) / 256 * (long long)a.rows;
  const unsigned grid = (unsigned)std::min((warps + 7) / 8, (long long)num_sms * 64);
  if (vec) dropout_kernel<TX, TY, true><<<grid, 256, 0, st>>>(a);
  else dropout_kernel<TX, TY, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int num_sms, cudaStream_t st) {
  if (a.rows <= 0 || a.cols <= 0) return cudaSuccess;
  const bool vec = rows_on_16(a.x, a.x_stride, a.x_bf16 ? 2 : 4) && rows_on_16(a.y, a.y_stride, a.y_bf16 ? 2 : 4) &&
                   (!a.residual || rows_on_16(a.residual, a.res_stride, a.y_bf16 ? 2 : 4));
  if (a.x_bf16) {
    if (a.y_bf16) launch<__nv_bfloat16, __nv_bfloat16>(a, vec, num_sms, st);
    else launch<__nv_bfloat16, float>(a, vec, num_sms, st);
  } else {
    if (a.y_bf16) launch<float, __nv_bfloat16>(a, vec, num_sms, st);
    else launch<float, float>(a, vec, num_sms, st);
  }
  return cudaGetLastError();
}

}  // namespace esm
