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

// ---- the gradient of larger batches: tokens sorted by id, then summed in pieces of 32 ----
// Sorting: one cluster of eight blocks sorts (id, token) by id, token order kept (least significant digit
// first), so that every id's tokens stand together in rising order.  A warp owns a contiguous stretch of the
// list; per pass it counts its digits (lanes with equal digits find each other by match, so one lane writes
// each count and no atomics order anything), the blocks exchange their counts through distributed shared
// memory, and every warp then knows where each of its digits goes.  Up to 8 bits per pass: one pass for
// 256 ids, two for 65536.  The rest of the grid meanwhile clears d_table.
constexpr int kSortBlocks = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 8, kBins = 1 << kDigitBits;

struct SortArgs {
  uint2 *list, *other;  // (id, token); the last pass writes list
  int* valid;      // tokens with a row
  int passes, digit_bits;
};

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __cluster_dims__(kSortBlocks, 1, 1) __launch_bounds__(kSortThreads)
    embed_sort_kernel(const EmbedArgs a, const SortArgs s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x >= kSortBlocks) {
    // (d_table is zeroed in 16-byte steps where it allows them)
    const size_t n = (size_t)a.vocab * a.cols, step = (size_t)(gridDim.x - kSortBlocks) * kSortThreads;
    const size_t first = (size_t)(blockIdx.x - kSortBlocks) * kSortThreads + tid;
    const size_t n4 = (reinterpret_cast<uintptr_t>(a.d_table) & 15) == 0 ? n / 4 : 0;
    for (size_t i = first; i < n4; i += step) reinterpret_cast<float4*>(a.d_table)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (size_t i = 4 * n4 + first; i < n; i += step) a.d_table[i] = 0.f;
    return;
  }
  __shared__ int hist[kSortWarps * kBins];  // counts, then next positions
  __shared__ int block_count[kBins];
  __shared__ int warp_total[kSortWarps];
  const int rank = (int)cluster_ctarank(), bins = 1 << s.digit_bits;
  int* mine = hist + warp * kBins;
  int n = a.tokens;
  for (int pass = 0; pass < s.passes; ++pass) {
    const uint2* src = (s.passes - pass) & 1 ? s.other : s.list;
    uint2* dst = (s.passes - pass) & 1 ? s.list : s.other;
    const int shift = pass * s.digit_bits;
    const int stretch = ((n + kSortBlocks * kSortWarps - 1) / (kSortBlocks * kSortWarps) + 31) & ~31;
    const long long begin = (long long)(rank * kSortWarps + warp) * stretch;
    const int end = (int)min((long long)n, begin + stretch);
    for (int d = lane; d < bins; d += 32) mine[d] = 0;
    __syncwarp();
    auto item = [&](int i) -> uint2 {  // an id of -1: none
      if (i >= end) return make_uint2(0xffffffffu, 0);
      if (pass) return __ldcg(src + i);
      return make_uint2((uint32_t)checked_id(a, i, true), (uint32_t)i);
    };
    for (long long i0 = begin; i0 < end; i0 += 32) {
      const uint2 v = item((int)i0 + lane);
      const int d = v.x == 0xffffffffu ? kBins : (int)(v.x >> shift) & (bins - 1);
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      if (d < kBins && lane == __ffs(peers) - 1) mine[d] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    // counts of the warps before, and the block's
    if (tid < bins) {
      int sum = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = hist[w * kBins + tid];
        hist[w * kBins + tid] = sum;
        sum += c;
      }
      block_count[tid] = sum;
    }
    __syncwarp();
    cluster_sync();
    int total = 0, before = 0;
    if (tid < bins) {
#pragma unroll
      for (int r = 0; r < kSortBlocks; ++r) {
        const int c = ld_cluster(map_to_rank(block_count + tid, r));
        total += c;
        if (r < rank) before += c;
      }
    }
    // where each digit starts: exclusive scan of the totals
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int lower = 0, all = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = warp_total[w];
      if (w < warp) lower += c;
      all += c;
    }
    if (tid < bins) {
      const int start = lower + incl - total + before;
      for (int w = 0; w < kSortWarps; ++w) hist[w * kBins + tid] += start;
    }
    __syncthreads();
    for (long long i0 = begin; i0 < end; i0 += 32) {
      const uint2 v = item((int)i0 + lane);
      const int d = v.x == 0xffffffffu ? kBins : (int)(v.x >> shift) & (bins - 1);
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      const int ahead = __popc(peers & ((1u << lane) - 1));
      if (d < kBins) dst[mine[d] + ahead] = v;
      __syncwarp();
      if (d < kBins && ahead == 0) mine[d] += __popc(peers);
      __syncwarp();
    }
    n = all;
    __syncwarp();
    // (also: no block counts again, or leaves, while another still reads its counts)
    cluster_sync();
  }
  if (rank == 0 && tid == 0) *s.valid = n;
}

// Sums of 32 consecutive places of the sorted list and 256 columns by one warp.  An id whose tokens all lie
// within the piece is written at once; of an id that goes on over the piece's border the piece keeps its part:
// part[piece][0] for one that began before, part[piece][1] for one that begins here and goes on.
constexpr int kPiece = 32;

template <typename TO, bool VEC>
__global__ void __launch_bounds__(256) embed_grad_pieces_kernel(const EmbedArgs a, const uint2* __restrict__ list,
                                                                const int* __restrict__ valid, float* __restrict__ part) {
  constexpr int kAhead = 4;  // rows in flight
  const PhiloxState ps = philox_state(a.mask);
  const int lane = threadIdx.x & 31, n = *valid;
  const int spans = (a.cols + 255) / 256;
  const long long per_row = (a.cols + 7) / 8, total = (long long)spans * ((n + kPiece - 1) / kPiece);
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
    const int piece = (int)(i / spans), c0 = (int)(i - (long long)piece * spans) * 256, left = min(256, a.cols - c0);
    const int p0 = piece * kPiece, count = min(kPiece, n - p0);
    const uint2 own = lane < count ? list[p0 + lane] : make_uint2(0xffffffffu, 0);
    const float own_scale = lane < count ? token_scale(a, (int)own.y) * a.mask.scale : 0.f;
    const int before = p0 > 0 ? (int)list[p0 - 1].x : -1, after = p0 + kPiece < n ? (int)list[p0 + kPiece].x : -1;
    int id = (int)__shfl_sync(0xffffffffu, own.x, 0);
    float acc[8] = {};
    auto leave = [&](bool last) {
      const bool from_before = id == before, goes_on = last && id == after;
      if (from_before || goes_on) {
        span_store<VEC>(part + ((size_t)piece * 2 + (from_before ? 0 : 1)) * a.cols + c0, left, lane, acc);
        return;
      }
      float* dst = a.d_table + (size_t)id * a.cols + c0;
      if (a.accumulate) {
        float old[8];
        span_load<VEC>(dst, left, lane, old);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += old[k];
      }
      span_store<VEC>(dst, left, lane, acc);
    };
    for (int j0 = 0; j0 < count; j0 += kAhead) {
      float g[kAhead][8];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int t = (int)__shfl_sync(0xffffffffu, own.y, j0 + j);
        if (j0 + j < count) span_load<VEC>(static_cast<const TO*>(a.out) + (size_t)t * a.out_stride + c0, left, lane, g[j]);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int t = (int)__shfl_sync(0xffffffffu, own.y, j0 + j), v = (int)__shfl_sync(0xffffffffu, own.x, j0 + j);
        const float f = __shfl_sync(0xffffffffu, own_scale, j0 + j);
        if (j0 + j >= count) break;
        if (v != id) {
          leave(false);
          id = v;
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = 0.f;
        }
        const uint32_t keep = span_keep<VEC>(a.mask, ps, (unsigned long long)(t * per_row + c0 / 8), lane);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += keep >> k & 1u ? g[j][k] * f : 0.f;
      }
    }
    leave(true);
  }
}

// Ids that cross borders: one block per piece in which such an id begins and 256 columns; its warps add
// the pieces' parts in turn, then the warps' sums are added in order.
template <bool VEC>
__global__ void __launch_bounds__(256) embed_grad_join_kernel(const EmbedArgs a, const uint2* __restrict__ list,
                                                              const int* __restrict__ valid,
                                                              const float* __restrict__ part) {
  __shared__ float sums[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = *valid;
  const int spans = (a.cols + 255) / 256, pieces = (n + kPiece - 1) / kPiece;
  for (long long i = blockIdx.x; i < (long long)spans * pieces; i += gridDim.x) {
    const int piece = (int)(i / spans), c0 = (int)(i - (long long)piece * spans) * 256, left = min(256, a.cols - c0);
    const int p0 = piece * kPiece;
    if (p0 + kPiece >= n) continue;
    const uint32_t id = list[p0 + kPiece - 1].x;
    if (list[p0 + kPiece].x != id || (p0 > 0 && list[p0 - 1].x == id)) continue;
    // the pieces that begin with this id: they follow one another
    int more = 0;
    for (int k0 = piece + 1;; k0 += 32) {
      const int k = k0 + lane;
      const int same = __popc(__ballot_sync(0xffffffffu, k < pieces && list[(size_t)min(k, pieces - 1) * kPiece].x == id));
      more += same;
      if (same < 32) break;
    }
    float acc[8] = {}, v[8];
    for (int k = warp; k <= more; k += 8) {
      span_load<VEC>(part + ((size_t)(piece + k) * 2 + (k ? 0 : 1)) * a.cols + c0, left, lane, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[warp][32 * e + lane] = acc[e];
    __syncthreads();
    if (warp == 0) {
      float* dst = a.d_table + (size_t)id * a.cols + c0;
      if (a.accumulate) span_load<VEC>(dst, left, lane, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += sums[w][32 * e + lane];
        v[e] = a.accumulate ? v[e] + s : s;
      }
      span_store<VEC>(dst, left, lane, v);
    }
    __syncthreads();
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

// Few tokens: a search through all of them for every id is one launch.
bool direct(int tokens, int vocab) { return tokens <= 512 && (long long)vocab * tokens <= 1 << 18; }

struct GradWorkspace {
  size_t list[2], valid, part, total;
};
GradWorkspace grad_workspace(int tokens, int cols) {
  const size_t T = (size_t)std::max(tokens, 1), pieces = (T + kPiece - 1) / kPiece;
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  GradWorkspace w;
  w.list[0] = 0;
  w.list[1] = w.list[0] + up(sizeof(uint2) * T);
  w.valid = w.list[1] + up(sizeof(uint2) * T);
  w.part = w.valid + 256;
  w.total = w.part + up(sizeof(float) * pieces * 2 * cols);
  return w;
}

template <typename TO, bool VEC>
cudaError_t launch_grad(const EmbedArgs& a, void* workspace, int num_sms, cudaStream_t st) {
  const long long spans = (a.cols + 255) / 256;
  if (direct(a.tokens, a.vocab)) {
    embed_grad_kernel<TO, VEC><<<warps_grid(spans * a.vocab, num_sms), 256, 0, st>>>(a);
    return cudaGetLastError();
  }
  const GradWorkspace w = grad_workspace(a.tokens, a.cols);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SortArgs s;
  s.list = reinterpret_cast<uint2*>(ws + w.list[0]);
  s.other = reinterpret_cast<uint2*>(ws + w.list[1]);
  s.valid = reinterpret_cast<int*>(ws + w.valid);
  int bits = 1;
  while (bits < 31 && (1ll << bits) < a.vocab) ++bits;
  s.passes = (bits + kDigitBits - 1) / kDigitBits;
  s.digit_bits = (bits + s.passes - 1) / s.passes;
  float* part = reinterpret_cast<float*>(ws + w.part);
  int clear = 0;  // blocks that clear d_table: a few KB each at least
  if (!a.accumulate) {
    const size_t bytes = 4 * (size_t)a.vocab * a.cols;
    clear = (int)std::min((bytes + (1 << 17) - 1) >> 17, (size_t)num_sms * 2);
    clear = (clear + kSortBlocks - 1) / kSortBlocks * kSortBlocks;
  }
  embed_sort_kernel<<<kSortBlocks + clear, kSortThreads, 0, st>>>(a, s);
  const long long pieces = (a.tokens + kPiece - 1) / kPiece;
  embed_grad_pieces_kernel<TO, VEC><<<warps_grid(spans * pieces, num_sms), 256, 0, st>>>(a, s.list, s.valid, part);
  const unsigned join = (unsigned)std::min(spans * pieces, (long long)num_sms * 32);
  embed_grad_join_kernel<VEC><<<join, 256, 0, st>>>(a, s.list, s.valid, part);
  return cudaGetLastError();
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

size_t embed_grad_workspace_bytes(int tokens, int vocab, int cols) {
  return direct(tokens, vocab) ? 256 : grad_workspace(tokens, cols).total;
}

cudaError_t launch_embed_grad(const EmbedArgs& a, void* workspace, int num_sms, cudaStream_t st) {
  const bool vec = rows_on_16(a.d_table, a.cols, 4) && rows_on_16(a.out, a.out_stride, a.out_bf16 ? 2 : 4);
  if (a.out_bf16)
    return vec ? launch_grad<__nv_bfloat16, true>(a, workspace, num_sms, st)
               : launch_grad<__nv_bfloat16, false>(a, workspace, num_sms, st);
  return vec ? launch_grad<float, true>(a, workspace, num_sms, st) : launch_grad<float, false>(a, workspace, num_sms, st);
}

}  // namespace esm
