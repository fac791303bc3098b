// Dropout whose mask is drawn again wherever it is needed and never stored (see dropout.cuh):
//   y = [residual +] keep(r, c) * scale * x
// The gradient is the same call on dy.
//
// Bound by memory: x (and the residual) read once, y written once.  16384 x 5120 in bfloat16: 54.7 us, 6.1 TB/s,
// 92 % of a copy's rate; the generator's issue slots, some two thirds of all, hide behind it.  The launch bound fits
// bfloat16; with float32 operands the aligned kernel spills 108 to 360 bytes: bfloat16 to float32 81 us (floor 75), float32
// to bfloat16 92 (75), float32 to float32 157 (100).
#include <algorithm>

#include "dropout.cuh"
#include "internal.h"

namespace esm {
namespace {

// Blocks of eight elements in the order of the rows: a thread takes four of them, 256 apart, and has all its
// loads on the way before it draws the first bits; the four calls of the generator share its round keys.
// DENSE: rows follow each other without a gap, so a block's place is its number.
constexpr int kBlocks = 4;

template <typename TX, typename TY, bool DENSE>
__global__ void __launch_bounds__(256, 4) dropout_kernel(const DropoutArgs a, const FastDiv per_row, long long total) {
  const PhiloxState ps = philox_state(a.mask);
  const TX* xs = static_cast<const TX*>(a.x);
  const TY* rs = static_cast<const TY*>(a.residual);
  TY* ys = static_cast<TY*>(a.y);
  const long long first = (long long)blockIdx.x * (256 * kBlocks) + threadIdx.x;
  Raw8<TX> x[kBlocks];
  Raw8<TY> r[kBlocks];
  long long row[kBlocks];
  int col[kBlocks], left[kBlocks];
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const long long b = first + j * 256;
    if (DENSE) {
      // (one row of all elements, in units of eight)
      row[j] = b * 8;
      col[j] = 0;
      left[j] = b < total ? 8 : 0;
    } else {
      row[j] = total <= INT32_MAX ? (long long)div_by((uint32_t)min(b, total), per_row) : b / per_row.d;
      col[j] = (int)(b - row[j] * per_row.d) * 8;
      left[j] = b < total ? a.cols - col[j] : 0;
    }
    const long long xi = DENSE ? row[j] : row[j] * a.x_stride + col[j];
    const long long ri = DENSE ? row[j] : row[j] * a.res_stride + col[j];
    if (left[j] > 0) x[j].load(xs + xi, left[j]);
    if (left[j] > 0 && rs) r[j].load(rs + ri, left[j]);
  }
  const uint64_t scale = f2_both(a.mask.scale);
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const uint4 w = drop_words(a.mask, ps, (unsigned long long)(first + j * 256));
    Pairs v;
    x[j].get(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], scale);
    keep(w, ps, v);
    if (rs) {
      Pairs add;
      r[j].get(add);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2_add(v[i], add[i]);
    }
    const long long yi = DENSE ? row[j] : row[j] * a.y_stride + col[j];
    if (left[j] > 0) span_store<true>(ys + yi, left[j], 0, v);
  }
}

// Rows whose eights are not aligned: one warp per 256 columns of a row (8191 x 1283 out of rows of 1288, added to a
// float32 residual: 20.6 us, 5.1 TB/s).
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) dropout_rows_kernel(const DropoutArgs a, const FastDiv spans, long long total) {
  const PhiloxState ps = philox_state(a.mask);
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5), per_row = (a.cols + 7) / 8;
  if (i >= total) return;
  const long long row = total <= INT32_MAX ? (long long)div_by((uint32_t)i, spans) : i / spans.d;
  const int c0 = (int)(i - row * spans.d) * 256, left = a.cols - c0;
  Pairs x, r;
  span_load<false>(static_cast<const TX*>(a.x) + row * a.x_stride + c0, left, lane, x);
  if (a.residual) span_load<false>(static_cast<const TY*>(a.residual) + row * a.res_stride + c0, left, lane, r);
  const uint4 own = drop_words(a.mask, ps, (unsigned long long)(row * per_row + c0 / 8 + lane));
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = f2_mul(x[k], f2_both(a.mask.scale));
  keep(span_words<false>(a.mask, own, lane), ps, x);
  if (a.residual) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = f2_add(x[k], r[k]);
  }
  span_store<false>(static_cast<TY*>(a.y) + row * a.y_stride + c0, left, lane, x);
}

template <typename TX, typename TY>
cudaError_t launch(const DropoutArgs& a, bool vec, bool dense, cudaStream_t st) {
  if (vec) {
    const int per_row = (a.cols + 7) / 8;
    const long long total = (long long)a.rows * per_row, grid = (total + 256 * kBlocks - 1) / (256 * kBlocks);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (dense) dropout_kernel<TX, TY, true><<<(unsigned)grid, 256, 0, st>>>(a, fast_div(per_row), total);
    else dropout_kernel<TX, TY, false><<<(unsigned)grid, 256, 0, st>>>(a, fast_div(per_row), total);
  } else {
    const int spans = (a.cols + 255) / 256;
    const long long total = (long long)a.rows * spans, grid = (total + 7) / 8;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    dropout_rows_kernel<TX, TY><<<(unsigned)grid, 256, 0, st>>>(a, fast_div(spans), total);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t st) {
  if (a.rows <= 0 || a.cols <= 0) return cudaSuccess;
  const bool vec = rows_on_eights(a.x, a.x_stride, a.x_bf16 ? 2 : 4) && rows_on_eights(a.y, a.y_stride, a.y_bf16 ? 2 : 4) &&
                   (!a.residual || rows_on_eights(a.residual, a.res_stride, a.y_bf16 ? 2 : 4));
  const bool dense = a.cols % 8 == 0 && (a.rows == 1 || (a.x_stride == a.cols && a.y_stride == a.cols &&
                                                         (!a.residual || a.res_stride == a.cols)));
  using bf16 = __nv_bfloat16;
  if (a.x_bf16) return a.y_bf16 ? launch<bf16, bf16>(a, vec, dense, st) : launch<bf16, float>(a, vec, dense, st);
  return a.y_bf16 ? launch<float, bf16>(a, vec, dense, st) : launch<float, float>(a, vec, dense, st);
}

}  // namespace esm
